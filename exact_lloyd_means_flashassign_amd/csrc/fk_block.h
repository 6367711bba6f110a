// Launchers of the expert-block operators: layer norm, top-k router, products
// with an epilogue (one weight or one per expert), weighted combine.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fk {

// ---- layer norm (fk_norm.hip) ----------------------------------------------
// Partial rows (2 d fp32 each) that the backward pass needs for dw and db.
int norm_partials(int64_t rows, int d);
hipError_t launch_layer_norm(int dtype, int wdtype, const void *X, int64_t ldx, int64_t rows, int d, const void *w,
                             const void *b, float eps, void *Y, int64_t ldy, float *mean, float *rstd, hipStream_t s);
hipError_t launch_layer_norm_bwd(int dtype, int wdtype, const void *dY, int64_t ldd, const void *X, int64_t ldx,
                                 int64_t rows, int d, const float *mean, const float *rstd, const void *w, void *dX,
                                 int64_t lddx, void *dw, void *db, float *part, hipStream_t s);
// out0[c] (c < split) and out1[c - split] = the sums of P partial rows of ld
// fp32 columns, added in a fixed order and rounded to dtype
hipError_t launch_sum_partials(const float *part, int P, int64_t ld, int64_t split, void *out0, void *out1, int dtype,
                               hipStream_t s);

// ---- router (fk_route.hip) ---------------------------------------------------
// Workgroups of the forward pass, each leaving one partial row: column sums of
// the probabilities and of lse^2, counts and live rows.
int route_blocks(int64_t T, int E);
size_t route_scratch_bytes(int64_t T, int E);
hipError_t launch_route(int dtype, const void *logits, int64_t ldl, int64_t T, int E, int k, int norm,
                        const uint8_t *valid, int32_t *ids, float *gates, int32_t *counts, float *losses,
                        int32_t *live, void *scratch, hipStream_t s);
hipError_t launch_route_bwd(int dtype, const void *logits, int64_t ldl, int64_t T, int E, int k, int norm,
                            const uint8_t *valid, const int32_t *ids, const int32_t *counts, const int32_t *live,
                            const float *d_gates, const float *d_losses, void *d_logits, hipStream_t s);

// ---- combine (fk_combine.hip) --------------------------------------------------
hipError_t launch_combine(int dtype, const void *Y, int64_t rows, int k, int d, const float *gates, const void *R,
                          int64_t ldr, void *out, int64_t ldo, hipStream_t s);
hipError_t launch_combine_bwd(int dtype, const void *dOut, int64_t ldo, const void *Y, int64_t rows, int k, int d,
                              const float *gates, void *dY, float *dgates, hipStream_t s);

// ---- products (fk_linear.hip) ---------------------------------------------------
struct LinearShape {
    int dtype, ydtype, act, bias_f32;
    bool grouped, by_slots;             // by_slots: rows of X and dY are taken by a slot list
    int G, share;
    int64_t M, N, K;                    // positions, columns of Y, length of the sum
    int64_t ldx, ldw, ldr, ldy, ldz, lddx;  // row strides
};
struct LinearPlan {
    int64_t M;
    int G;
    bool few, tiled, pad_x, pad_w, sort_x, make_dz;
    int tile, splits, tile_w, splits_w;
    int64_t grad_tiles;
    size_t xpad, wpad, part, dz, colsum, total;
};
struct LinearBufs {
    const void *X, *W, *bias, *R, *dY, *Zin;
    const int32_t *slots, *offsets;
    void *Y, *Z, *dX, *dW, *db;
};
LinearPlan plan_linear(const LinearShape &h, bool backward);
hipError_t launch_linear(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, void *ws, hipStream_t s);
hipError_t launch_linear_bwd(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, void *ws, hipStream_t s);

}  // namespace fk
