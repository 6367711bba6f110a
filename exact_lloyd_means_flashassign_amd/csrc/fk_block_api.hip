// Host side of the expert-block operators: argument checks, workspace layout
// and launches on the caller's stream.  Declared in include/fk.h.
#include <cmath>

#include "fk.h"
#include "fk_block.h"
#include "fk_host.h"
#include "fk_internal.h"
#include "fk_rows.h"

using namespace fk;

namespace {

fk_status check_dtype(int32_t t, const char *what) {
    if (!known_dtype(t)) return fail(FK_ERR_INVALID_ARG, "unknown %s %d", what, (int)t);
    return FK_OK;
}

fk_status check_rows(int64_t rows, int64_t d) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(FK_ERR_INVALID_ARG, "rows=%lld outside [0, 2^31-1]", (long long)rows);
    if (d < 1 || d > FK_MAX_WIDTH)
        return fail(FK_ERR_INVALID_ARG, "row width %lld outside [1, %d]", (long long)d, FK_MAX_WIDTH);
    return FK_OK;
}

// A matrix argument: there when there are rows, its rows not overlapping, and
// starting on its elements.
fk_status check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size, const char *name) {
    if (rows > 0 && p == nullptr) return fail(FK_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, size)) return fail(FK_ERR_INVALID_ARG, "%s must be aligned to its elements", name);
    if (ld < cols)
        return fail(FK_ERR_INVALID_ARG, "%s has row stride %lld, under its %lld columns", name, (long long)ld,
                    (long long)cols);
    if (ld > ((int64_t)1 << 40)) return fail(FK_ERR_INVALID_ARG, "%s has row stride %lld", name, (long long)ld);
    return FK_OK;
}

// What an argument takes up: `bytes` from p on, of a matrix only `width` out of
// every `pitch`.
struct Span {
    const void *p;
    size_t bytes;
    const char *name;
    size_t width = 0, pitch = 0;
};
Span matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, size_t size, const char *name) {
    return {p, rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * size : 0, name, (size_t)cols * size,
            (size_t)ld * size};
}

// Whether two spans have a byte in common.  Matrices of one pitch may lie in
// each other's gaps: column slices of one buffer.
bool share_bytes(const Span &a, const Span &b) {
    if (!overlap(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    const size_t far = pb >= pa ? (pb - pa) % a.pitch : a.pitch - 1 - (pa - pb - 1) % a.pitch;  // b's rows after a's
    return far < a.width || far + b.width > a.pitch;
}

// No output overlaps an input or another output.
fk_status check_apart(const Span *outs, int nout, const Span *ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        if (outs[i].p == nullptr || outs[i].bytes == 0) continue;
        for (int j = 0; j < nin + i; ++j) {
            const Span &o = j < nin ? ins[j] : outs[j - nin];
            if (o.p == nullptr || o.bytes == 0) continue;
            if (share_bytes(outs[i], o))
                return fail(FK_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, o.name);
        }
    }
    return FK_OK;
}

#define FK_CHECK(expr)                        \
    do {                                      \
        const fk_status st_ = (expr);         \
        if (st_ != FK_OK) return st_;         \
    } while (0)

fk_status check_norm(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d) {
    FK_CHECK(check_dtype(dtype, "element type"));
    FK_CHECK(check_dtype(wdtype, "parameter type"));
    if (wdtype != dtype && wdtype != FK_F32)
        return fail(FK_ERR_UNSUPPORTED, "parameters must be of the rows' type or fp32");
    return check_rows(rows, d);
}

}  // namespace

extern "C" {

fk_status fk_layer_norm(int32_t dtype, int32_t wdtype, const void *X, int64_t ldx, int64_t rows, int32_t d,
                        const void *weight, const void *bias, float eps, void *Y, int64_t ldy, float *mean,
                        float *rstd, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_norm(dtype, wdtype, rows, d));
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(FK_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", (double)eps);
    const size_t sz = dtype_size(dtype), wsz = dtype_size(wdtype);
    FK_CHECK(check_matrix(X, rows, d, ldx, sz, "X"));
    FK_CHECK(check_matrix(Y, rows, d, ldy, sz, "Y"));
    if (!aligned(weight, wsz) || !aligned(bias, wsz) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(FK_ERR_INVALID_ARG, "weight, bias, mean and rstd must be aligned to their elements");
    const bool in_place = X == Y && ldx == ldy;
    const Span ins[] = {matrix(in_place ? nullptr : X, rows, d, ldx, sz, "X"), {weight, d * wsz, "weight"},
                        {bias, d * wsz, "bias"}};
    const Span outs[] = {matrix(Y, rows, d, ldy, sz, "Y"), {mean, (size_t)rows * 4, "mean"}, {rstd, (size_t)rows * 4, "rstd"}};
    FK_CHECK(check_apart(outs, 3, ins, 3));
    FK_CHECK(check_device());
    if (rows == 0) return FK_OK;
    FK_TRY(launch_layer_norm(dtype, wdtype, X, ldx, rows, d, weight, bias, eps, Y, ldy, mean, rstd, (hipStream_t)stream),
           "layer norm");
    return FK_OK;
}

size_t fk_layer_norm_backward_workspace_size(int64_t rows, int32_t d) {
    if (rows < 0 || rows > INT32_MAX || d < 1 || d > FK_MAX_WIDTH) return 0;
    return align_up((size_t)norm_partials(rows, d) * 2 * (size_t)d * 4 + 1, 256);
}

fk_status fk_layer_norm_backward(int32_t dtype, int32_t wdtype, const void *dY, int64_t lddy, const void *X,
                                 int64_t ldx, int64_t rows, int32_t d, const float *mean, const float *rstd,
                                 const void *weight, void *dX, int64_t lddx, void *dweight, void *dbias,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_norm(dtype, wdtype, rows, d));
    const size_t sz = dtype_size(dtype), wsz = dtype_size(wdtype);
    FK_CHECK(check_matrix(dY, rows, d, lddy, sz, "dY"));
    FK_CHECK(check_matrix(X, rows, d, ldx, sz, "X"));
    FK_CHECK(check_matrix(dX, rows, d, lddx, sz, "dX"));
    if (rows > 0 && (mean == nullptr || rstd == nullptr))
        return fail(FK_ERR_INVALID_ARG, "mean and rstd must not be NULL");
    if (!aligned(weight, wsz) || !aligned(dweight, wsz) || !aligned(dbias, wsz) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(FK_ERR_INVALID_ARG, "weight, mean, rstd, dweight and dbias must be aligned to their elements");
    const bool in_place = dX == dY && lddx == lddy;
    if (in_place && rows > 0 && d > 8192)
        return fail(FK_ERR_UNSUPPORTED, "dX may be dY only for rows of at most 8192 elements");
    const Span ins[] = {matrix(in_place ? nullptr : dY, rows, d, lddy, sz, "dY"), matrix(X, rows, d, ldx, sz, "X"),
                        {weight, d * wsz, "weight"}, {mean, (size_t)rows * 4, "mean"}, {rstd, (size_t)rows * 4, "rstd"}};
    const Span outs[] = {matrix(dX, rows, d, lddx, sz, "dX"), {dweight, d * wsz, "dweight"}, {dbias, d * wsz, "dbias"}};
    FK_CHECK(check_apart(outs, 3, ins, 5));
    FK_CHECK(check_workspace(workspace, workspace_bytes, fk_layer_norm_backward_workspace_size(rows, d)));
    FK_CHECK(check_device());
    FK_TRY(launch_layer_norm_bwd(dtype, wdtype, dY, lddy, X, ldx, rows, d, mean, rstd, weight, dX, lddx, dweight, dbias,
                                 (float *)workspace, (hipStream_t)stream),
           "layer norm backward");
    return FK_OK;
}

}  // extern "C"

namespace {
fk_status check_route(int32_t dtype, const void *logits, int64_t ldl, int64_t T, int32_t E, int32_t k, int32_t norm) {
    FK_CHECK(check_dtype(dtype, "element type"));
    if (T < 0 || T > INT32_MAX) return fail(FK_ERR_INVALID_ARG, "T=%lld outside [0, 2^31-1]", (long long)T);
    if (E < 1 || E > FK_MAX_EXPERTS) return fail(FK_ERR_INVALID_ARG, "E=%d outside [1, %d]", (int)E, FK_MAX_EXPERTS);
    if (k < 1 || k > E || k > FK_MAX_ROUTE_K)
        return fail(FK_ERR_INVALID_ARG, "k=%d outside [1, min(E, %d)]", (int)k, FK_MAX_ROUTE_K);
    if (T * k > INT32_MAX) return fail(FK_ERR_INVALID_ARG, "T k = %lld slots, over 2^31-1", (long long)(T * k));
    if (norm != FK_GATES_CHOSEN && norm != FK_GATES_ALL) return fail(FK_ERR_INVALID_ARG, "unknown gate norm %d", (int)norm);
    return check_matrix(logits, T, E, ldl, dtype_size(dtype), "logits");
}
}  // namespace

extern "C" {

size_t fk_route_workspace_size(int64_t T, int32_t E) {
    if (T < 0 || T > INT32_MAX || E < 1 || E > FK_MAX_EXPERTS) return 0;
    return align_up(route_scratch_bytes(T, E), 256);
}

fk_status fk_route(int32_t dtype, const void *logits, int64_t ldl, int64_t T, int32_t E, int32_t k, int32_t gate_norm,
                   const uint8_t *valid, int32_t *ids, float *gates, int32_t *counts, float *losses, int32_t *live,
                   void *workspace, size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_route(dtype, logits, ldl, T, E, k, gate_norm));
    if (T > 0 && (ids == nullptr || gates == nullptr))
        return fail(FK_ERR_INVALID_ARG, "ids and gates must not be NULL");
    if (counts == nullptr || losses == nullptr || live == nullptr)
        return fail(FK_ERR_INVALID_ARG, "counts, losses and live must not be NULL");
    if (!aligned(ids, 4) || !aligned(gates, 4) || !aligned(counts, 4) || !aligned(losses, 4) || !aligned(live, 4))
        return fail(FK_ERR_INVALID_ARG, "ids, gates, counts, losses and live must be aligned to 4 bytes");
    const Span ins[] = {matrix(logits, T, E, ldl, dtype_size(dtype), "logits"), {valid, (size_t)T, "valid"}};
    const Span outs[] = {{ids, (size_t)T * k * 4, "ids"}, {gates, (size_t)T * k * 4, "gates"},
                         {counts, (size_t)E * 4, "counts"}, {losses, 8, "losses"}, {live, 4, "live"}};
    FK_CHECK(check_apart(outs, 5, ins, 2));
    FK_CHECK(check_workspace(workspace, workspace_bytes, fk_route_workspace_size(T, E)));
    FK_CHECK(check_device());
    FK_TRY(launch_route(dtype, logits, ldl, T, E, k, gate_norm, valid, ids, gates, counts, losses, live, workspace,
                        (hipStream_t)stream),
           "router");
    return FK_OK;
}

fk_status fk_route_backward(int32_t dtype, const void *logits, int64_t ldl, int64_t T, int32_t E, int32_t k,
                            int32_t gate_norm, const uint8_t *valid, const int32_t *ids, const int32_t *counts,
                            const int32_t *live, const float *d_gates, const float *d_losses, void *d_logits,
                            void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_route(dtype, logits, ldl, T, E, k, gate_norm));
    if (T > 0 && ids == nullptr) return fail(FK_ERR_INVALID_ARG, "ids is NULL");
    if (counts == nullptr || live == nullptr) return fail(FK_ERR_INVALID_ARG, "counts and live must not be NULL");
    FK_CHECK(check_matrix(d_logits, T, E, E, dtype_size(dtype), "d_logits"));
    if (!aligned(ids, 4) || !aligned(counts, 4) || !aligned(live, 4) || !aligned(d_gates, 4) || !aligned(d_losses, 4))
        return fail(FK_ERR_INVALID_ARG, "ids, counts, live, d_gates and d_losses must be aligned to 4 bytes");
    const size_t sz = dtype_size(dtype);
    const Span ins[] = {matrix(logits, T, E, ldl, sz, "logits"), {valid, (size_t)T, "valid"}, {ids, (size_t)T * k * 4, "ids"},
                        {counts, (size_t)E * 4, "counts"}, {live, 4, "live"}, {d_gates, (size_t)T * k * 4, "d_gates"},
                        {d_losses, 8, "d_losses"}};
    const Span outs[] = {matrix(d_logits, T, E, E, sz, "d_logits")};
    FK_CHECK(check_apart(outs, 1, ins, 7));
    FK_CHECK(check_device());
    if (T == 0) return FK_OK;
    FK_TRY(launch_route_bwd(dtype, logits, ldl, T, E, k, gate_norm, valid, ids, counts, live, d_gates, d_losses,
                            d_logits, (hipStream_t)stream),
           "router backward");
    return FK_OK;
}

}  // extern "C"

namespace {

fk_status check_linear(const fk_linear_shape *h) {
    if (h == nullptr) return fail(FK_ERR_INVALID_ARG, "shape is NULL");
    FK_CHECK(check_dtype(h->dtype, "element type"));
    FK_CHECK(check_dtype(h->ydtype, "output type"));
    FK_CHECK(check_dtype(h->bias_dtype, "bias type"));
    if ((h->ydtype != h->dtype && h->ydtype != FK_F32) || (h->bias_dtype != h->dtype && h->bias_dtype != FK_F32))
        return fail(FK_ERR_UNSUPPORTED, "the output and the bias must be of the operands' type or fp32");
    if (h->act < FK_ACT_NONE || h->act > FK_ACT_SILU) return fail(FK_ERR_INVALID_ARG, "unknown activation %d", (int)h->act);
    if (h->M < 0 || h->M > INT32_MAX) return fail(FK_ERR_INVALID_ARG, "M=%lld outside [0, 2^31-1]", (long long)h->M);
    if (h->N < 1 || h->N > FK_MAX_WIDTH || h->K < 1 || h->K > FK_MAX_WIDTH)
        return fail(FK_ERR_INVALID_ARG, "N=%lld or K=%lld outside [1, %d]", (long long)h->N, (long long)h->K, FK_MAX_WIDTH);
    if (h->groups < 0 || h->groups > FK_MAX_GROUPS)
        return fail(FK_ERR_INVALID_ARG, "groups=%d outside [0, %d]", (int)h->groups, FK_MAX_GROUPS);
    if (h->share < 1 || (h->groups == 0 && h->share != 1))
        return fail(FK_ERR_INVALID_ARG, "share=%d must be >= 1, and 1 without groups", (int)h->share);
    if (h->M % h->share != 0)
        return fail(FK_ERR_INVALID_ARG, "M=%lld slots are no multiple of share=%d", (long long)h->M, (int)h->share);
    return FK_OK;
}

LinearShape shape_of(const fk_linear_shape *h, bool by_slots) {
    LinearShape s{};
    s.dtype = h->dtype, s.ydtype = h->ydtype, s.act = h->act, s.bias_f32 = h->bias_dtype == FK_F32;
    s.grouped = h->groups > 0, s.by_slots = by_slots, s.G = h->groups > 0 ? h->groups : 1, s.share = h->share;
    s.M = h->M, s.N = h->N, s.K = h->K;
    s.ldx = h->ldx, s.ldw = h->ldw, s.ldr = h->ldr, s.ldy = h->ldy, s.ldz = h->ldpre, s.lddx = h->K;
    return s;
}

fk_status check_slots(const fk_linear_shape *h, const int32_t *slots, const int32_t *offsets) {
    if (h->groups > 0 && offsets == nullptr) return fail(FK_ERR_INVALID_ARG, "offsets is NULL");
    if (h->groups > 0 && slots == nullptr && h->share != 1)
        return fail(FK_ERR_INVALID_ARG, "share=%d needs a slot list", (int)h->share);
    if (h->groups == 0 && (slots != nullptr || offsets != nullptr))
        return fail(FK_ERR_INVALID_ARG, "slots and offsets need groups > 0");
    if (!aligned(slots, 4) || !aligned(offsets, 4))
        return fail(FK_ERR_INVALID_ARG, "slots and offsets must be aligned to 4 bytes");
    return FK_OK;
}

// Rows of whole 16-byte chunks are read chunk by chunk; others element by
// element, wherever they start.
fk_status check_start(const void *p, int64_t cols, int64_t ld, size_t size, const char *name) {
    const int64_t chunk = 16 / (int64_t)size;
    if (cols % chunk == 0 && ld % chunk == 0 && !aligned(p, 16))
        return fail(FK_ERR_INVALID_ARG, "%s must be 16-byte aligned, its rows being whole 16-byte chunks", name);
    return FK_OK;
}

}  // namespace

extern "C" {

size_t fk_linear_workspace_size(const fk_linear_shape *shape, int32_t backward) {
    // (a list only ever adds to what is needed)
    if (check_linear(shape) != FK_OK) return 0;
    return plan_linear(shape_of(shape, shape->groups > 0 && !(backward & 2)), backward & 1).total;
}

fk_status fk_linear(const fk_linear_shape *shape, const void *X, const void *W, const void *bias,
                    const void *residual, const int32_t *slots, const int32_t *offsets, void *Y, void *pre,
                    void *workspace, size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_linear(shape));
    const LinearShape h = shape_of(shape, slots != nullptr);
    const size_t sz = dtype_size(h.dtype), ysz = dtype_size(h.ydtype), bsz = dtype_size(shape->bias_dtype);
    const int64_t xr = h.M / h.share;
    FK_CHECK(check_matrix(X, xr, h.K, h.ldx, sz, "X"));
    FK_CHECK(check_matrix(W, (int64_t)h.G * h.N, h.K, h.ldw, sz, "W"));
    FK_CHECK(check_matrix(Y, h.M, h.N, h.ldy, ysz, "Y"));
    if (residual) FK_CHECK(check_matrix(residual, h.M, h.N, h.ldr, sz, "residual"));
    if (pre) FK_CHECK(check_matrix(pre, h.M, h.N, h.ldz, sz, "pre"));
    FK_CHECK(check_start(X, h.K, h.ldx, sz, "X"));
    FK_CHECK(check_start(W, h.K, h.ldw, sz, "W"));
    if (!aligned(bias, bsz)) return fail(FK_ERR_INVALID_ARG, "bias must be aligned to its elements");
    FK_CHECK(check_slots(shape, slots, offsets));
    const bool in_place = residual == Y && h.ldr == h.ldy && h.dtype == h.ydtype;
    const Span ins[] = {matrix(X, xr, h.K, h.ldx, sz, "X"), matrix(W, (int64_t)h.G * h.N, h.K, h.ldw, sz, "W"),
                        {bias, (size_t)h.G * h.N * bsz, "bias"},
                        matrix(in_place ? nullptr : residual, h.M, h.N, h.ldr, sz, "residual"),
                        {slots, (size_t)h.M * 4, "slots"}, {offsets, (size_t)(h.G + 1) * 4, "offsets"}};
    const Span outs[] = {matrix(Y, h.M, h.N, h.ldy, ysz, "Y"), matrix(pre, h.M, h.N, h.ldz, sz, "pre")};
    FK_CHECK(check_apart(outs, 2, ins, 6));
    const LinearPlan p = plan_linear(h, false);
    FK_CHECK(check_workspace(workspace, workspace_bytes, p.total));
    FK_CHECK(check_device());
    if (h.M == 0) return FK_OK;
    LinearBufs b{};
    b.X = X, b.W = W, b.bias = bias, b.R = residual, b.slots = slots, b.offsets = offsets, b.Y = Y, b.Z = pre;
    FK_TRY(launch_linear(h, p, b, workspace, (hipStream_t)stream), "product");
    return FK_OK;
}

fk_status fk_linear_backward(const fk_linear_shape *shape, const void *dY, const void *X, const void *W,
                             const void *pre, const int32_t *slots, const int32_t *offsets, void *dX, void *dW,
                             void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_linear(shape));
    const LinearShape h = shape_of(shape, slots != nullptr);
    const size_t sz = dtype_size(h.dtype), ysz = dtype_size(h.ydtype), bsz = dtype_size(shape->bias_dtype);
    const int64_t xr = h.M / h.share, wr = (int64_t)h.G * h.N;
    FK_CHECK(check_matrix(dY, h.M, h.N, h.ldy, ysz, "dY"));
    if (dW) FK_CHECK(check_matrix(X, xr, h.K, h.ldx, sz, "X"));
    if (dX) FK_CHECK(check_matrix(W, wr, h.K, h.ldw, sz, "W"));
    if (h.act != FK_ACT_NONE) FK_CHECK(check_matrix(pre, h.M, h.N, h.ldz, sz, "pre"));
    FK_CHECK(check_start(dY, h.N, h.ldy, ysz, "dY"));
    FK_CHECK(check_start(X, h.K, h.ldx, sz, "X"));
    FK_CHECK(check_start(W, h.K, h.ldw, sz, "W"));
    if (!aligned(dX, sz) || !aligned(dW, sz) || !aligned(dbias, bsz))
        return fail(FK_ERR_INVALID_ARG, "dX, dW and dbias must be aligned to their elements");
    FK_CHECK(check_slots(shape, slots, offsets));
    const Span ins[] = {matrix(dY, h.M, h.N, h.ldy, ysz, "dY"), matrix(X, xr, h.K, h.ldx, sz, "X"),
                        matrix(W, wr, h.K, h.ldw, sz, "W"), matrix(pre, h.M, h.N, h.ldz, sz, "pre"),
                        {slots, (size_t)h.M * 4, "slots"}, {offsets, (size_t)(h.G + 1) * 4, "offsets"}};
    const Span outs[] = {matrix(dX, h.M, h.K, h.K, sz, "dX"), matrix(dW, wr, h.K, h.K, sz, "dW"),
                         {dbias, (size_t)wr * bsz, "dbias"}};
    FK_CHECK(check_apart(outs, 3, ins, 6));
    const LinearPlan p = plan_linear(h, true);
    FK_CHECK(check_workspace(workspace, workspace_bytes, p.total));
    FK_CHECK(check_device());
    LinearBufs b{};
    b.X = X, b.W = W, b.dY = dY, b.Zin = pre, b.slots = slots, b.offsets = offsets, b.dX = h.M > 0 ? dX : nullptr;
    b.dW = dW, b.db = dbias;
    FK_TRY(launch_linear_bwd(h, p, b, workspace, (hipStream_t)stream), "product backward");
    return FK_OK;
}

}  // extern "C"

namespace {
fk_status check_combine(int32_t dtype, int64_t rows, int32_t k, int32_t d) {
    FK_CHECK(check_dtype(dtype, "element type"));
    FK_CHECK(check_rows(rows, d));
    if (k < 1 || k > FK_MAX_ROUTE_K) return fail(FK_ERR_INVALID_ARG, "k=%d outside [1, %d]", (int)k, FK_MAX_ROUTE_K);
    if (rows * k > INT32_MAX) return fail(FK_ERR_INVALID_ARG, "rows k = %lld slots, over 2^31-1", (long long)(rows * k));
    return FK_OK;
}
}  // namespace

extern "C" {

fk_status fk_combine(int32_t dtype, const void *Y, int64_t rows, int32_t k, int32_t d, const float *gates,
                     const void *residual, int64_t ldr, void *out, int64_t ldo, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_combine(dtype, rows, k, d));
    const size_t sz = dtype_size(dtype);
    FK_CHECK(check_matrix(Y, rows, d, d, sz, "Y"));
    FK_CHECK(check_matrix(out, rows, d, ldo, sz, "out"));
    if (residual) FK_CHECK(check_matrix(residual, rows, d, ldr, sz, "residual"));
    if (!aligned(gates, 4)) return fail(FK_ERR_INVALID_ARG, "gates must be aligned to 4 bytes");
    const bool in_place = residual == out && ldr == ldo;
    const Span ins[] = {matrix(Y, rows * k, d, d, sz, "Y"), {gates, (size_t)rows * k * 4, "gates"},
                        matrix(in_place ? nullptr : residual, rows, d, ldr, sz, "residual")};
    const Span outs[] = {matrix(out, rows, d, ldo, sz, "out")};
    FK_CHECK(check_apart(outs, 1, ins, 3));
    FK_CHECK(check_device());
    if (rows == 0) return FK_OK;
    FK_TRY(launch_combine(dtype, Y, rows, k, d, gates, residual, ldr, out, ldo, (hipStream_t)stream), "combine");
    return FK_OK;
}

fk_status fk_combine_backward(int32_t dtype, const void *dOut, int64_t lddo, const void *Y, int64_t rows, int32_t k,
                              int32_t d, const float *gates, void *dY, float *dgates, void *stream) {
    g_err[0] = 0;
    FK_CHECK(check_combine(dtype, rows, k, d));
    const size_t sz = dtype_size(dtype);
    FK_CHECK(check_matrix(dOut, rows, d, lddo, sz, "dOut"));
    FK_CHECK(check_matrix(dY, rows, d, d, sz, "dY"));
    if (dgates != nullptr) FK_CHECK(check_matrix(Y, rows, d, d, sz, "Y"));
    if (!aligned(gates, 4) || !aligned(dgates, 4)) return fail(FK_ERR_INVALID_ARG, "gates and dgates must be aligned to 4 bytes");
    const Span ins[] = {matrix(dOut, rows, d, lddo, sz, "dOut"), matrix(Y, rows * k, d, d, sz, "Y"),
                        {gates, (size_t)rows * k * 4, "gates"}};
    const Span outs[] = {matrix(dY, rows * k, d, d, sz, "dY"), {dgates, (size_t)rows * k * 4, "dgates"}};
    FK_CHECK(check_apart(outs, 2, ins, 3));
    FK_CHECK(check_device());
    if (rows == 0) return FK_OK;
    FK_TRY(launch_combine_bwd(dtype, dOut, lddo, Y, rows, k, d, gates, dY, dgates, (hipStream_t)stream),
           "combine backward");
    return FK_OK;
}

}  // extern "C"
