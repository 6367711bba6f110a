// Layer norm for gfx950, forward and backward.
//
//   mu = mean_j x_j,  r = 1/sqrt(mean_j (x_j - mu)^2 + eps),  xh = (x - mu) r
//   y = xh w + b
//   g = dy w,  dx = r (g - mean(g) - xh mean(g xh)),  dw = sum dy xh,  db = sum dy
//
// Bound by memory: the forward pass reads a row and writes one, the backward
// pass reads two and writes one, at a handful of fp32 operations an element.
// A row is held in the registers of a team (a wave up to 2048 elements, a
// workgroup of 256 threads up to 8192), so it is read once although the
// variance is taken around the mean; longer rows are read again, from cache.
// Teams walk the rows with the grid's stride, the next row's loads in flight
// while this one is summed, and keep the weights (forward) and the columns'
// sums of dw and db (backward) in registers; the sums leave as one partial row
// for each workgroup and are added in a fixed order by a second kernel, so
// there are no atomics and results are bitwise reproducible.  All sums are
// fp32.
//
// Measured at 32749 x 4096 in bf16: forward 97 us (5.5 TB/s), backward 157 us
// (5.1 TB/s) and 7 us for the partial rows, where a copy of 1 GiB runs at 5.1.
// A few rows take 4 us on the device, less than the launch.  Rows that are no
// whole 16-byte chunks go element by element: 32749 x 4095 144 and 212 us.  Rows
// past 8192 elements are read three times: 8191 x 16384 forward 475 us (1.1
// TB/s of what has to move), backward 490 and 161 for the columns.
#include "fk.h"
#include "fk_block.h"
#include "fk_internal.h"
#include "fk_rows.h"

namespace fk {

namespace {

constexpr int kNormMaxHeld = 8192;  // longest row held in registers

struct NormArgs {
    const void *X, *dY, *w, *b;
    const float *mean_in, *rstd_in;
    void *Y;
    float *mean, *rstd, *part;
    int64_t rows, ldx, ldy, ldd;  // row strides of X, the output, dY
    int d, wf32;
    float eps;
};

// A thread's elements of a row: NCH chunks of V, chunk c at (c TEAM + t) V.
template <typename T, int V, int TEAM, int NCH>
__global__ __launch_bounds__(256) void k_layer_norm(NormArgs a) {
    __shared__ float sred[2][8];
    constexpr int RPB = 256 / TEAM;
    const int t = threadIdx.x % TEAM;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TEAM;
    const int d = a.d;
    const T *X = (const T *)a.X;
    T *Y = (T *)a.Y;
    float w[NCH][V], b[NCH][V];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int j = (c * TEAM + t) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[c][i] = 1.0f;
            b[c][i] = 0.0f;
        }
        if (j < d) {
            if (a.w) load_param<T, V>(a.w, a.wf32, j, w[c]);
            if (a.b) load_param<T, V>(a.b, a.wf32, j, b[c]);
        }
    }
    Chunk<T, V> x[NCH];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (c * TEAM + t) * V;
            if (r < a.rows && j < d) x[c].load(X + r * a.ldx + j);
            else x[c].zero();
        }
    };
    fetch(row);
    const float inv_d = 1.0f / (float)d;
    // every team of a workgroup runs the same number of rounds (barriers)
    for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step, row += step) {
        float v[NCH][V];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[c][i] = (float)x[c].e[i];
                s[0] += v[c][i];
            }
        fetch(row + step);
        team_sum<TEAM, 1>(s, sred[0]);
        const float mu = s[0] * inv_d;
        float q[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const bool in = (c * TEAM + t) * V < d;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[c][i] = in ? v[c][i] - mu : 0.0f;
                q[0] += v[c][i] * v[c][i];
            }
        }
        team_sum<TEAM, 1>(q, sred[1]);
        const float r = 1.0f / sqrtf(q[0] * inv_d + a.eps);
        if (row < a.rows) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int j = (c * TEAM + t) * V;
                if (j < d) {
                    Chunk<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.e[i] = (T)(v[c][i] * r * w[c][i] + b[c][i]);
                    o.store(Y + row * a.ldy + j);
                }
            }
            if (t == 0) {
                if (a.mean) a.mean[row] = mu;
                if (a.rstd) a.rstd[row] = r;
            }
        }
    }
}

template <typename T, int V, int TEAM, int NCH>
__global__ __launch_bounds__(256) void k_layer_norm_bwd(NormArgs a) {
    __shared__ float sred[2][8];
    constexpr int RPB = 256 / TEAM;
    const int t = threadIdx.x % TEAM;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TEAM;
    const int d = a.d;
    const T *X = (const T *)a.X, *dY = (const T *)a.dY;
    T *dX = (T *)a.Y;
    float w[NCH][V], sw[NCH][V], sb[NCH][V];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int j = (c * TEAM + t) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[c][i] = 1.0f;
            sw[c][i] = sb[c][i] = 0.0f;
        }
        if (j < d && a.w) load_param<T, V>(a.w, a.wf32, j, w[c]);
    }
    Chunk<T, V> x[NCH], g[NCH];
    float mu = 0.0f, r = 0.0f;
    auto fetch = [&](int64_t rw) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int j = (c * TEAM + t) * V;
            if (rw < a.rows && j < d) {
                x[c].load(X + rw * a.ldx + j);
                g[c].load(dY + rw * a.ldd + j);
            } else {
                x[c].zero();
                g[c].zero();
            }
        }
        mu = rw < a.rows ? a.mean_in[rw] : 0.0f;
        r = rw < a.rows ? a.rstd_in[rw] : 0.0f;
    };
    fetch(row);
    const float inv_d = 1.0f / (float)d;
    int round = 0;
    for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step, row += step, round ^= 1) {
        float xh[NCH][V], gw[NCH][V];
        float s[2] = {0.0f, 0.0f};
        const float r0 = r, mu0 = mu;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            // elements past the row are zero in g but not in (0 - mu) r
            const bool in = (c * TEAM + t) * V < d;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gy = (float)g[c].e[i];
                xh[c][i] = in ? ((float)x[c].e[i] - mu0) * r0 : 0.0f;
                gw[c][i] = gy * w[c][i];
                sw[c][i] += gy * xh[c][i];
                sb[c][i] += gy;
                s[0] += gw[c][i];
                s[1] += gw[c][i] * xh[c][i];
            }
        }
        fetch(row + step);
        team_sum<TEAM, 2>(s, sred[round]);
        const float c1 = s[0] * inv_d, c2 = s[1] * inv_d;
        if (row < a.rows) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int j = (c * TEAM + t) * V;
                if (j < d) {
                    Chunk<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.e[i] = (T)(r0 * (gw[c][i] - c1 - xh[c][i] * c2));
                    o.store(dX + row * a.ldy + j);
                }
            }
        }
    }
    if (a.part == nullptr) return;
    float *out = a.part + (size_t)blockIdx.x * 2 * d;
    if constexpr (TEAM == 64) {
        // the four waves' columns, added in wave order
        __shared__ float scol[2][64 * NCH * V];
        for (int wv = 0; wv < 4; ++wv) {
            if (threadIdx.x / 64 == wv) {
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int k = (c * V + i) * 64 + t;
                        scol[0][k] = (wv ? scol[0][k] : 0.0f) + sw[c][i];
                        scol[1][k] = (wv ? scol[1][k] : 0.0f) + sb[c][i];
                    }
            }
            __syncthreads();
        }
        if (threadIdx.x >= 64) return;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sw[c][i] = scol[0][(c * V + i) * 64 + t];
                sb[c][i] = scol[1][(c * V + i) * 64 + t];
            }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int j = (c * TEAM + t) * V;
        if (j < d) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                out[j + i] = sw[c][i];
                out[d + j + i] = sb[c][i];
            }
        }
    }
}

// Rows longer than a team holds: a workgroup per row, which it reads again
// for each step (a row of 16-bit elements stays in cache well past 2^20).
template <typename T>
__global__ __launch_bounds__(256) void k_layer_norm_long(NormArgs a) {
    __shared__ float sred[2][8];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = (const T *)a.X + row * a.ldx;
        T *y = (T *)a.Y + row * a.ldy;
        float s[1] = {0.0f};
        for (int j = threadIdx.x; j < a.d; j += 256) s[0] += (float)x[j];
        team_sum<256, 1>(s, sred[0]);
        const float mu = s[0] / (float)a.d;
        float q[1] = {0.0f};
        for (int j = threadIdx.x; j < a.d; j += 256) {
            const float v = (float)x[j] - mu;
            q[0] += v * v;
        }
        team_sum<256, 1>(q, sred[1]);
        const float r = 1.0f / sqrtf(q[0] / (float)a.d + a.eps);
        for (int j = threadIdx.x; j < a.d; j += 256) {
            float w[1] = {1.0f}, b[1] = {0.0f};
            if (a.w) load_param<T, 1>(a.w, a.wf32, j, w);
            if (a.b) load_param<T, 1>(a.b, a.wf32, j, b);
            y[j] = (T)(((float)x[j] - mu) * r * w[0] + b[0]);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_layer_norm_bwd_long(NormArgs a) {
    __shared__ float sred[2][8];
    int round = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, round ^= 1) {
        const T *x = (const T *)a.X + row * a.ldx, *dy = (const T *)a.dY + row * a.ldd;
        T *dx = (T *)a.Y + row * a.ldy;
        const float mu = a.mean_in[row], r = a.rstd_in[row];
        float s[2] = {0.0f, 0.0f};
        for (int j = threadIdx.x; j < a.d; j += 256) {
            float w[1] = {1.0f};
            if (a.w) load_param<T, 1>(a.w, a.wf32, j, w);
            const float g = (float)dy[j] * w[0];
            s[0] += g;
            s[1] += g * ((float)x[j] - mu) * r;
        }
        team_sum<256, 2>(s, sred[round]);
        const float c1 = s[0] / (float)a.d, c2 = s[1] / (float)a.d;
        for (int j = threadIdx.x; j < a.d; j += 256) {
            float w[1] = {1.0f};
            if (a.w) load_param<T, 1>(a.w, a.wf32, j, w);
            dx[j] = (T)(r * ((float)dy[j] * w[0] - c1 - ((float)x[j] - mu) * r * c2));
        }
    }
}

// The long rows' columns: 64 columns and one run of rows a workgroup, its
// four waves taking every fourth row.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_cols_long(NormArgs a, int64_t run) {
    __shared__ float sm[2][4][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t j = (int64_t)blockIdx.x * 64 + lane;
    const int64_t r0 = blockIdx.y * run, r1 = r0 + run < a.rows ? r0 + run : a.rows;
    float sw = 0.0f, sb = 0.0f;
    if (j < a.d) {
        for (int64_t r = r0 + wv; r < r1; r += 4) {
            const float g = (float)((const T *)a.dY)[r * a.ldd + j];
            sw += g * (((float)((const T *)a.X)[r * a.ldx + j] - a.mean_in[r]) * a.rstd_in[r]);
            sb += g;
        }
    }
    sm[0][wv][lane] = sw;
    sm[1][wv][lane] = sb;
    __syncthreads();
    if (wv == 0 && j < a.d) {
        float *out = a.part + (size_t)blockIdx.y * 2 * a.d;
        out[j] = sm[0][0][lane] + sm[0][1][lane] + sm[0][2][lane] + sm[0][3][lane];
        out[a.d + j] = sm[1][0][lane] + sm[1][1][lane] + sm[1][2][lane] + sm[1][3][lane];
    }
}

// out[c] = sum_p part[p, c] over P partial rows of ld fp32 columns: 16 columns
// a workgroup, 16 threads down each.  Columns [0, split) go to out0, the rest
// to out1 (either may be NULL).
template <typename T>
__global__ __launch_bounds__(256) void k_sum_partials(const float *__restrict__ part, int P, int64_t ld, int64_t split,
                                                      void *out0, void *out1, int f32) {
    __shared__ float sm[16][17];
    const int col = threadIdx.x & 15, down = threadIdx.x >> 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    float s = 0.0f;
    if (c < ld) {
#pragma unroll 8
        for (int p = down; p < P; p += 16) s += part[(size_t)p * ld + c];
    }
    sm[down][col] = s;
    __syncthreads();
    if (down == 0 && c < ld) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += sm[i][col];
        void *o = c < split ? out0 : out1;
        const int64_t at = c < split ? c : c - split;
        if (o != nullptr) {
            if (f32) ((float *)o)[at] = t;
            else ((T *)o)[at] = (T)t;
        }
    }
}

// Workgroups of a backward pass: two for every CU (a partial row each), fewer
// when the rows run out.
int bwd_blocks(int64_t rows, int d) {
    const int64_t per = d <= 2048 ? 4 : 1;
    const int64_t need = cdiv(rows, per);
    return (int)(need < 512 ? need : 512);
}
constexpr int kLongRuns = 64;

template <typename T, int V, bool BWD>
hipError_t launch_held(const NormArgs &a, hipStream_t s) {
    constexpr int C = 8 / V;  // chunks that hold 8 elements
#define FK_NORM(TEAM, NCH)                                                                                    \
    do {                                                                                                      \
        if constexpr (BWD) {                                                                                  \
            k_layer_norm_bwd<T, V, TEAM, NCH><<<bwd_blocks(a.rows, a.d), 256, 0, s>>>(a);                     \
        } else {                                                                                              \
            const int64_t need = cdiv(a.rows, 256 / TEAM);                                                    \
            k_layer_norm<T, V, TEAM, NCH><<<(unsigned)(need < 2048 ? need : 2048), 256, 0, s>>>(a);           \
        }                                                                                                     \
    } while (0)
    if (a.d <= 512) FK_NORM(64, C);
    else if (a.d <= 1024) FK_NORM(64, 2 * C);
    else if (a.d <= 2048) FK_NORM(64, 4 * C);
    else if (a.d <= 4096) FK_NORM(256, 2 * C);
    else FK_NORM(256, 4 * C);
#undef FK_NORM
    return hipGetLastError();
}

template <typename T, bool BWD>
hipError_t launch_norm(const NormArgs &a, bool wide, hipStream_t s) {
    if (a.d > kNormMaxHeld) {
        const unsigned grid = (unsigned)(a.rows < 4096 ? a.rows : 4096);
        if constexpr (BWD) {
            k_layer_norm_bwd_long<T><<<grid, 256, 0, s>>>(a);
            if (a.part != nullptr) {
                const int64_t run = cdiv(a.rows, norm_partials(a.rows, a.d));
                k_norm_cols_long<T><<<dim3((unsigned)cdiv(a.d, 64), (unsigned)norm_partials(a.rows, a.d)), 256, 0, s>>>(a, run);
            }
        } else {
            k_layer_norm_long<T><<<grid, 256, 0, s>>>(a);
        }
        return hipGetLastError();
    }
    if (wide) return launch_held<T, 16 / (int)sizeof(T), BWD>(a, s);
    return launch_held<T, 1, BWD>(a, s);
}

// 16-byte chunks need rows and parameters that start on 16 bytes and whole
// chunks in a row.
bool chunked(const NormArgs &a, int size) {
    const int v = 16 / size;
    auto ok = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
    return a.d % v == 0 && a.ldx % v == 0 && a.ldy % v == 0 && a.ldd % v == 0 && ok(a.X) && ok(a.Y) && ok(a.dY) &&
           ok(a.w) && ok(a.b);
}

template <bool BWD>
hipError_t dispatch_norm(int dtype, const NormArgs &a, hipStream_t s) {
    const bool wide = chunked(a, (int)dtype_size(dtype));
    switch (dtype) {
    case FK_F32: return launch_norm<float, BWD>(a, wide, s);
    case FK_BF16: return launch_norm<__bf16, BWD>(a, wide, s);
    default: return launch_norm<_Float16, BWD>(a, wide, s);
    }
}

}  // namespace

int norm_partials(int64_t rows, int d) {
    if (d <= kNormMaxHeld) return bwd_blocks(rows, d);
    return (int)(rows < kLongRuns ? rows : kLongRuns);
}

hipError_t launch_sum_partials(const float *part, int P, int64_t ld, int64_t split, void *out0, void *out1, int dtype,
                               hipStream_t s) {
    const unsigned grid = (unsigned)cdiv(ld, 16);
    if (dtype == FK_BF16) k_sum_partials<__bf16><<<grid, 256, 0, s>>>(part, P, ld, split, out0, out1, 0);
    else if (dtype == FK_F16) k_sum_partials<_Float16><<<grid, 256, 0, s>>>(part, P, ld, split, out0, out1, 0);
    else k_sum_partials<float><<<grid, 256, 0, s>>>(part, P, ld, split, out0, out1, 1);
    return hipGetLastError();
}

hipError_t launch_layer_norm(int dtype, int wdtype, const void *X, int64_t ldx, int64_t rows, int d, const void *w,
                             const void *b, float eps, void *Y, int64_t ldy, float *mean, float *rstd, hipStream_t s) {
    NormArgs a{};
    a.X = X, a.w = w, a.b = b, a.Y = Y, a.mean = mean, a.rstd = rstd;
    a.rows = rows, a.ldx = ldx, a.ldy = ldy, a.d = d, a.wf32 = wdtype == FK_F32, a.eps = eps;
    return dispatch_norm<false>(dtype, a, s);
}

hipError_t launch_layer_norm_bwd(int dtype, int wdtype, const void *dY, int64_t ldd, const void *X, int64_t ldx,
                                 int64_t rows, int d, const float *mean, const float *rstd, const void *w, void *dX,
                                 int64_t lddx, void *dw, void *db, float *part, hipStream_t s) {
    NormArgs a{};
    a.X = X, a.dY = dY, a.w = w, a.Y = dX, a.mean_in = mean, a.rstd_in = rstd, a.part = dw || db ? part : nullptr;
    a.rows = rows, a.ldx = ldx, a.ldd = ldd, a.ldy = lddx, a.d = d, a.wf32 = wdtype == FK_F32;
    hipError_t e = rows > 0 ? dispatch_norm<true>(dtype, a, s) : hipSuccess;
    if (e != hipSuccess || a.part == nullptr) return e;
    return launch_sum_partials(part, norm_partials(rows, d), 2 * (int64_t)d, d, dw, db, wdtype, s);
}

}  // namespace fk
