// The weighted sum of a row's expert outputs for gfx950, and its gradients.
//
//   out[t] = R[t] + sum_j g[t, j] Y[t k + j]
//   dY[t k + j] = g[t, j] dOut[t],   dg[t, j] = dOut[t] . Y[t k + j]
//
// Bound by memory: k rows read for one written (forward), k read and k
// written (backward).  The slots of a row lie next to each other, so the sum
// is a stream; the k rows are added in slot order in fp32 and rounded once.
// In the backward pass a team (a wave up to 2048 elements, a workgroup beyond)
// holds dOut's row in registers, reads each of the k rows once and writes its
// gradient on the way; the dot products of eight slots share one reduction.
// A gate of zero leaves its slot's row unread (forward) or writes zeros
// (backward, where dg still needs the row): a slot without an expert may hold
// anything.
//
// Measured at 16411 rows of 4 slots by 4096 in bf16 with a residual: forward
// 155 us (5.2 TB/s), backward 206 us (5.9 TB/s).  Rows that are no whole 16-byte
// chunks go element by element, each load waited for: by 4095 596 and 621 us.
#include "fk.h"
#include "fk_block.h"
#include "fk_internal.h"
#include "fk_rows.h"

namespace fk {

namespace {

constexpr int kCombineMaxHeld = 8192;

struct CombineArgs {
    const void *Y, *R, *dOut;
    const float *gates;
    void *out;
    float *dgates;
    int64_t rows, ldr, ldo;  // row strides of R, and of out or dOut
    int d, k;
};

// TX lanes across a row's chunks, 256 / TX rows a workgroup.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a, int lx) {
    const int tx = threadIdx.x & ((1 << lx) - 1), ty = threadIdx.x >> lx;
    const int rpb = 256 >> lx;
    const int nch = a.d / V;
    const T *Y = (const T *)a.Y, *R = (const T *)a.R;
    for (int64_t row = (int64_t)blockIdx.x * rpb + ty; row < a.rows; row += (int64_t)gridDim.x * rpb) {
        for (int c = blockIdx.y * (1 << lx) + tx; c < nch; c += gridDim.y << lx) {
            float s[V];
            Chunk<T, V> y;
            y.zero();
            if (R) y.load(R + row * a.ldr + (int64_t)c * V);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = (float)y.e[i];
            const T *p = Y + (row * a.k * (int64_t)nch + c) * V;
#pragma unroll 4
            for (int j = 0; j < a.k; ++j) {
                const float g = a.gates ? a.gates[row * a.k + j] : 1.0f;
                Chunk<T, V> v;
                v.zero();
                if (g != 0.0f) v.load(p + (int64_t)j * a.d);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += g * (float)v.e[i];
            }
            Chunk<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.e[i] = (T)s[i];
            o.store((T *)a.out + row * a.ldo + (int64_t)c * V);
        }
    }
}

constexpr int kDots = 8;  // slots that share one reduction

template <typename T, int V, int TEAM, int NCH>
__global__ __launch_bounds__(256) void k_combine_bwd(CombineArgs a) {
    __shared__ float sred[2][4 * kDots];
    constexpr int RPB = 256 / TEAM;
    const int t = threadIdx.x % TEAM;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int round = 0;
    for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step) {
        // a team past the last row goes through the barriers on no data
        const int64_t row = base + threadIdx.x / TEAM;
        const bool on = row < a.rows;
        Chunk<T, V> g[NCH];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (c * TEAM + t) * V;
            if (on && j < a.d) g[c].load((const T *)a.dOut + row * a.ldo + j);
            else g[c].zero();
        }
        for (int j0 = 0; j0 < a.k; j0 += kDots, round ^= 1) {
            float dot[kDots];
#pragma unroll
            for (int q = 0; q < kDots; ++q) {
                dot[q] = 0.0f;
                if (!on || j0 + q >= a.k) continue;
                const float w = a.gates ? a.gates[row * a.k + j0 + q] : 1.0f;
                const int64_t at = (row * a.k + j0 + q) * a.d;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const int j = (c * TEAM + t) * V;
                    if (j >= a.d) continue;
                    Chunk<T, V> y, o;
                    y.zero();
                    if (a.dgates) y.load((const T *)a.Y + at + j);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float v = (float)g[c].e[i];
                        dot[q] += v * (float)y.e[i];
                        o.e[i] = (T)(w == 0.0f ? 0.0f : w * v);
                    }
                    o.store((T *)a.out + at + j);
                }
            }
            if (a.dgates == nullptr) continue;
            team_sum<TEAM, kDots>(dot, sred[round]);
            if (on && t == 0) {
#pragma unroll
                for (int q = 0; q < kDots; ++q)
                    if (j0 + q < a.k) a.dgates[row * a.k + j0 + q] = dot[q];
            }
        }
    }
}

// Rows longer than a team holds: a workgroup per slot.
template <typename T>
__global__ __launch_bounds__(256) void k_combine_bwd_long(CombineArgs a) {
    __shared__ float sred[2][4];
    int round = 0;
    for (int64_t s = blockIdx.x; s < a.rows * a.k; s += gridDim.x, round ^= 1) {
        const T *g = (const T *)a.dOut + s / a.k * a.ldo, *y = (const T *)a.Y + s * a.d;
        T *o = (T *)a.out + s * a.d;
        const float w = a.gates ? a.gates[s] : 1.0f;
        float dot[1] = {0.0f};
        for (int j = threadIdx.x; j < a.d; j += 256) {
            const float v = (float)g[j];
            if (a.dgates) dot[0] += v * (float)y[j];
            o[j] = (T)(w == 0.0f ? 0.0f : w * v);
        }
        if (a.dgates == nullptr) continue;
        team_sum<256, 1>(dot, sred[round]);
        if (threadIdx.x == 0) a.dgates[s] = dot[0];
    }
}

template <typename T, int V>
hipError_t run_combine(const CombineArgs &a, hipStream_t s) {
    const int nch = a.d / V;
    int lx = 0;
    while ((1 << lx) < nch && lx < 8) ++lx;
    const int64_t bx = cdiv(a.rows, 256 >> lx);
    const int64_t by = cdiv(nch, 1 << lx);
    k_combine<T, V><<<dim3((unsigned)(bx < 65536 ? bx : 65536), (unsigned)(by < 1024 ? by : 1024)), 256, 0, s>>>(a, lx);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t run_combine_bwd(const CombineArgs &a, hipStream_t s) {
    constexpr int C = 8 / V;
    const int64_t per = a.d <= 2048 ? 4 : 1;
    const int64_t need = cdiv(a.rows, per);
    const unsigned grid = (unsigned)(need < 65536 ? need : 65536);
    if (a.d <= 512) k_combine_bwd<T, V, 64, C><<<grid, 256, 0, s>>>(a);
    else if (a.d <= 1024) k_combine_bwd<T, V, 64, 2 * C><<<grid, 256, 0, s>>>(a);
    else if (a.d <= 2048) k_combine_bwd<T, V, 64, 4 * C><<<grid, 256, 0, s>>>(a);
    else if (a.d <= 4096) k_combine_bwd<T, V, 256, 2 * C><<<grid, 256, 0, s>>>(a);
    else k_combine_bwd<T, V, 256, 4 * C><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

bool chunked(const CombineArgs &a, int size) {
    const int v = 16 / size;
    auto ok = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
    return a.d % v == 0 && a.ldr % v == 0 && a.ldo % v == 0 && ok(a.Y) && ok(a.R) && ok(a.dOut) && ok(a.out);
}

template <typename T>
hipError_t dispatch_combine(const CombineArgs &a, bool bwd, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool wide = chunked(a, (int)sizeof(T));
    if (!bwd) return wide ? run_combine<T, V>(a, s) : run_combine<T, 1>(a, s);
    if (a.d > kCombineMaxHeld) {
        const int64_t n = a.rows * a.k;
        k_combine_bwd_long<T><<<(unsigned)(n < 65536 ? n : 65536), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    return wide ? run_combine_bwd<T, V>(a, s) : run_combine_bwd<T, 1>(a, s);
}

hipError_t dispatch(int dtype, const CombineArgs &a, bool bwd, hipStream_t s) {
    switch (dtype) {
    case FK_F32: return dispatch_combine<float>(a, bwd, s);
    case FK_BF16: return dispatch_combine<__bf16>(a, bwd, s);
    default: return dispatch_combine<_Float16>(a, bwd, s);
    }
}

}  // namespace

hipError_t launch_combine(int dtype, const void *Y, int64_t rows, int k, int d, const float *gates, const void *R,
                          int64_t ldr, void *out, int64_t ldo, hipStream_t s) {
    CombineArgs a{};
    a.Y = Y, a.R = R, a.gates = gates, a.out = out, a.rows = rows, a.ldr = R ? ldr : 0, a.ldo = ldo, a.d = d, a.k = k;
    return dispatch(dtype, a, false, s);
}

hipError_t launch_combine_bwd(int dtype, const void *dOut, int64_t ldo, const void *Y, int64_t rows, int k, int d,
                              const float *gates, void *dY, float *dgates, hipStream_t s) {
    CombineArgs a{};
    a.Y = Y, a.dOut = dOut, a.gates = gates, a.out = dY, a.dgates = dgates, a.rows = rows, a.ldo = ldo, a.d = d, a.k = k;
    return dispatch(dtype, a, true, s);
}

}  // namespace fk
