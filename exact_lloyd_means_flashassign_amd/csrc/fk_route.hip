// Top-k router for gfx950 with per-expert counts, a balance loss and a z loss,
// and the gradient of all of them.
//
//   p = softmax(l) over the E experts, lse = log sum exp l
//   ids = the k largest logits, gates = softmax over those k, or their p
//   counts_e = slots that chose e,  f = counts / sum counts,  n = live rows
//   balance = E sum_e f_e (1/n) sum_t p_te,   z = (1/n) sum_t lse_t^2
// and, f being held constant (a count has no gradient),
//   dl = p (v - p.v) + dz 2 lse p / n + the gates' part,   v_e = dbalance E f_e / n
//   gates over the chosen: g (dg - g.dg);  gates = p: p_i (dg_i - sum_j p_j dg_j)
//
// Bound by memory at many rows (each logit read once a pass, its gradient
// written once) and by the launch at few.  A row belongs to a team of 2^m
// lanes, 8 consecutive experts a lane up to E = 512 (16 beyond), so a row's
// reductions are at most six lane exchanges and a lane meets the same experts
// in every row: the columns' sums and counts stay in its registers until the
// workgroup is done, and leave as one partial row, which a second kernel adds
// in a fixed order (a single workgroup finishes by itself).  No atomics.
//
// Selection compares logits as they are (no rounding), the lower index first
// on ties; a row that is not valid or has nothing above -inf is not live: its
// slots get id E and gate 0, and so do the slots of a live row past its last
// logit above -inf.  A NaN logit is never chosen; it makes its row's
// probabilities, and with them the losses, NaN.
#include "fk.h"
#include "fk_block.h"
#include "fk_internal.h"
#include "fk_rows.h"

namespace fk {

namespace {

constexpr int kRouteThreads = 1024;  // forward: one workgroup a CU, few partial rows
constexpr int kRouteMaxBlocks = 256;

struct RouteArgs {
    const void *logits;
    const uint8_t *valid;
    int32_t *ids, *counts, *live;
    float *gates, *losses;
    const int32_t *ids_in, *counts_in, *live_in;
    const float *d_gates, *d_losses;
    void *d_logits;
    float *part;  // [blocks][2 E + 2]: probability sums, lse^2, then (as int32) counts, live rows
    int64_t T, ldl;
    int E, k, norm, vec;
};

// e^x for x <= 0 to about an ulp: 2^(x log2 e) with the product's rounding
// error fed back in first order.
__device__ __forceinline__ float exp_neg(float x) {
    const float hi = x * 1.44269504f;
    const float lo = __builtin_fmaf(x, 1.44269504f, -hi) + x * 1.92596299e-8f;  // log2 e = their sum
    const float e = __builtin_amdgcn_exp2f(hi);
    // x = -inf: hi = -inf, lo = NaN, and the result is 0
    return e == 0.0f ? 0.0f : __builtin_fmaf(e, lo * 0.693147181f, e);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
    return lanes_sum<LPR>(v);
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_row(const RouteArgs &a, int64_t row, int col, bool on, float (&l)[VPL]) {
    constexpr int W = 16 / (int)sizeof(T);
    const T *p = (const T *)a.logits + row * a.ldl + col;
    if (a.vec) {
#pragma unroll
        for (int v = 0; v < VPL; v += W) {
            Chunk<T, W> c;
            const bool in = on && col + v < a.E;
            if (in) c.load(p + v);
#pragma unroll
            for (int i = 0; i < W; ++i) l[v + i] = in ? (float)c.e[i] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) l[v] = on && col + v < a.E ? (float)p[v] : -INFINITY;
    }
}

// The largest of the row's values that are not yet taken (bit v of `taken` for
// the lane's value v) and its expert, the lowest on ties; -1 if nothing above
// -inf is left.
template <int VPL, int LPR>
__device__ __forceinline__ void next_best(const float (&l)[VPL], uint32_t taken, int col, float &best, int &at) {
    best = -INFINITY;
    at = -1;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const bool better = !((taken >> v) & 1u) && l[v] > best;
        best = better ? l[v] : best;
        at = better ? col + v : at;
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
        const float ov = __shfl_xor(best, o, 64);
        const int oa = __shfl_xor(at, o, 64);
        const bool take = ov > best || (ov == best && (uint32_t)oa < (uint32_t)at);
        best = take ? ov : best;
        at = take ? oa : at;
    }
}

// The counts, live rows and losses from P partial rows, by one workgroup.
__device__ __forceinline__ void route_finish(const RouteArgs &a, int P, float *sm) {
    const int E = a.E, ld = 2 * E + 2;
    int *si = reinterpret_cast<int *>(sm);
    // columns [0, E]: fp32 (sums of p, sum of lse^2); (E, 2 E + 1]: counts and live rows.
    // Up to 16 runs of rows a column, added in run order.
    const int cols = ld;
    int down = kRouteThreads / 64;
    __shared__ float s_n[1];
    float bal = 0.0f;
    __shared__ float s_tot[16];
    float *colsum = sm + down * 64;
    for (int c0 = 0; c0 < cols; c0 += 64) {
        const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
        const int c = c0 + lane;
        float fs = 0.0f;
        int is = 0;
        if (c < cols) {
            for (int p = run; p < P; p += down) {
                const float v = a.part[(size_t)p * ld + c];
                if (c <= E) fs += v;
                else is += __float_as_int(v);
            }
        }
        __syncthreads();
        if (c <= E) sm[run * 64 + lane] = fs;
        else si[run * 64 + lane] = is;
        __syncthreads();
        if (run == 0 && c < cols) {
            if (c <= E) {
                float t = 0.0f;
                for (int r = 0; r < down; ++r) t += sm[r * 64 + lane];
                colsum[c] = t;
            } else {
                int t = 0;
                for (int r = 0; r < down; ++r) t += si[r * 64 + lane];
                reinterpret_cast<int *>(colsum)[c] = t;
                if (c < ld - 1) a.counts[c - E - 1] = t;
                else a.live[0] = t;
            }
        }
    }
    __syncthreads();
    const int *ci = reinterpret_cast<const int *>(colsum) + E + 1;
    // total slots and E sum_e counts_e psum_e
    float tot = 0.0f;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
        tot += (float)ci[e];
        bal += (float)ci[e] * colsum[e];
    }
    tot = lanes_sum<64>(tot);
    bal = lanes_sum<64>(bal);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        s_tot[threadIdx.x >> 6] = tot;
        sm[threadIdx.x >> 6] = bal;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f, b = 0.0f;
        for (int w = 0; w < kRouteThreads / 64; ++w) {
            t += s_tot[w];
            b += sm[w];
        }
        const float n = (float)(ci[E] > 0 ? ci[E] : 1);
        s_n[0] = n;
        a.losses[0] = (float)E * (b / (t > 0.0f ? t : 1.0f)) / n;
        a.losses[1] = colsum[E] / n;
    }
}

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a) {
    constexpr int RPB = kRouteThreads / LPR;  // rows a round
    constexpr int COLS = LPR * VPL;
    extern __shared__ float sm[];
    const int lane = threadIdx.x % LPR;
    const int col = lane * VPL;
    float psum[VPL];
    int cnt[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        psum[v] = 0.0f;
        cnt[v] = 0;
    }
    float zsum = 0.0f;
    int nlive = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < a.T; row += (int64_t)gridDim.x * RPB) {
        const bool valid = a.valid == nullptr || a.valid[row] != 0;
        float l[VPL];
        load_row<T, VPL>(a, row, col, valid, l);
        float m = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            m = fmaxf(m, l[v]);  // the larger of the two, NaN ignored
            nan = nan || l[v] != l[v];
        }
        m = row_max<LPR>(m);
        const float nans = row_sum<LPR>(nan ? 1.0f : 0.0f);
        const bool on = m != -INFINITY || nans > 0.0f;
        if (on) {
            float e[VPL], s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                e[v] = exp_neg(l[v] - m);
                s += e[v];
            }
            s = row_sum<LPR>(s);
            const float inv = 1.0f / s;
#pragma unroll
            for (int v = 0; v < VPL; ++v) psum[v] += e[v] * inv;
            if (lane == 0) {
                const float lse = m + logf(s);
                zsum += lse * lse;
                ++nlive;
            }
            // the k best in turn; the gates' sum over the chosen ones follows
            uint32_t taken = 0;
            float gsum = 0.0f;
            float mine = 0.0f;  // lane j of the team keeps gate j (several passes if k > LPR)
            for (int j0 = 0; j0 < a.k; j0 += LPR) {
                const int jn = a.k - j0 < LPR ? a.k - j0 : LPR;
                int myid = a.E;
                mine = 0.0f;
                for (int j = 0; j < jn; ++j) {
                    float best;
                    int at;
                    next_best<VPL, LPR>(l, taken, col, best, at);
                    const float ge = at >= 0 ? exp_neg(best - m) : 0.0f;
                    gsum += ge;
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        const bool here = at == col + v;
                        taken |= here ? 1u << v : 0u;
                        cnt[v] += here ? 1 : 0;
                    }
                    if (lane == j) {
                        mine = ge;
                        myid = at >= 0 ? at : a.E;
                    }
                }
                if (lane < jn) {
                    a.ids[row * a.k + j0 + lane] = myid;
                    a.gates[row * a.k + j0 + lane] = mine;  // scaled below
                }
            }
            const float scale = a.norm == FK_GATES_CHOSEN ? 1.0f / gsum : inv;
            // (a lane rewrites only what it wrote itself)
            for (int j = lane; j < a.k; j += LPR) {
                const float g = j >= a.k - (a.k - 1) % LPR - 1 ? mine : a.gates[row * a.k + j];
                a.gates[row * a.k + j] = g == 0.0f ? 0.0f : g * scale;
            }
        } else {
            for (int j = lane; j < a.k; j += LPR) {
                a.ids[row * a.k + j] = a.E;
                a.gates[row * a.k + j] = 0.0f;
            }
        }
    }
    // the teams' columns: lanes of a wave that own the same experts, then the
    // waves in order through LDS
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
#pragma unroll
        for (int o = LPR; o < 64; o <<= 1) {
            psum[v] += __shfl_xor(psum[v], o, 64);
            cnt[v] += __shfl_xor(cnt[v], o, 64);
        }
    }
    zsum = lanes_sum<64>(zsum);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) nlive += __shfl_xor(nlive, o, 64);
    constexpr int WV = kRouteThreads / 64;
    const int wv = threadIdx.x >> 6;
    __shared__ float s_z[WV];
    __shared__ int s_live[WV];
    int *si = reinterpret_cast<int *>(sm) + COLS;
    for (int w = 0; w < WV; ++w) {
        if (w == wv) {
            if ((threadIdx.x & 63) < LPR) {
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    sm[col + v] = (w ? sm[col + v] : 0.0f) + psum[v];
                    si[col + v] = (w ? si[col + v] : 0) + cnt[v];
                }
            }
            if ((threadIdx.x & 63) == 0) {
                s_z[w] = zsum;
                s_live[w] = nlive;
            }
        }
        __syncthreads();
    }
    float *out = a.part + (size_t)blockIdx.x * (2 * a.E + 2);
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        out[e] = sm[e];
        out[a.E + 1 + e] = __int_as_float(si[e]);
    }
    if (threadIdx.x == 0) {
        float z = 0.0f;
        int n = 0;
        for (int w = 0; w < WV; ++w) {
            z += s_z[w];
            n += s_live[w];
        }
        out[a.E] = z;
        out[2 * a.E + 1] = __int_as_float(n);
    }
    if (gridDim.x == 1) {
        __syncthreads();  // the partial row is read back by the same workgroup
        route_finish(a, 1, sm);
    }
}

__global__ __launch_bounds__(kRouteThreads) void k_route_finish(RouteArgs a, int P) {
    extern __shared__ float sm[];
    route_finish(a, P, sm);
}

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(256) void k_route_bwd(RouteArgs a) {
    constexpr int RPB = 256 / LPR;
    const int lane = threadIdx.x % LPR;
    const int col = lane * VPL;
    const float n = (float)(a.live_in[0] > 0 ? a.live_in[0] : 1);
    const float dbal = a.d_losses ? a.d_losses[0] : 0.0f, dz = a.d_losses ? a.d_losses[1] : 0.0f;
    // v_e = dbalance E f_e / n of this lane's experts
    float f[VPL];
    float tot = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        f[v] = col + v < a.E ? (float)a.counts_in[col + v] : 0.0f;
        tot += f[v];
    }
    tot = row_sum<LPR>(tot);
    const float fs = dbal * (float)a.E / (n * (tot > 0.0f ? tot : 1.0f));
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] *= fs;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < a.T; row += (int64_t)gridDim.x * RPB) {
        const bool valid = a.valid == nullptr || a.valid[row] != 0;
        float l[VPL], dl[VPL];
        load_row<T, VPL>(a, row, col, valid, l);
        float m = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            m = fmaxf(m, l[v]);
            nan = nan || l[v] != l[v];
            dl[v] = 0.0f;
        }
        m = row_max<LPR>(m);
        const float nans = row_sum<LPR>(nan ? 1.0f : 0.0f);
        if (m != -INFINITY || nans > 0.0f) {
            float e[VPL], s = 0.0f, pv = 0.0f;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                e[v] = exp_neg(l[v] - m);
                s += e[v];
                pv += e[v] * f[v];
            }
            s = row_sum<LPR>(s);
            pv = row_sum<LPR>(pv);
            const float inv = 1.0f / s;
            const float lse = m + logf(s);
            const float shift = dz * 2.0f * lse / n - pv * inv;
            // the gates: dg of the chosen experts, which are marked in `sel`
            float dg[VPL];
            uint32_t sel = 0;
#pragma unroll
            for (int v = 0; v < VPL; ++v) dg[v] = 0.0f;
            if (a.d_gates != nullptr) {
                for (int j = 0; j < a.k; ++j) {
                    const int at = a.ids_in[row * a.k + j] - col;
                    if ((unsigned)at < (unsigned)VPL) {
                        const float g = a.d_gates[row * a.k + j];
#pragma unroll
                        for (int v = 0; v < VPL; ++v) {
                            dg[v] = at == v ? g : dg[v];
                            sel |= at == v ? 1u << v : 0u;
                        }
                    }
                }
            }
            float es = 0.0f, in = 0.0f;
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                if ((sel >> v) & 1u) {
                    es += e[v];
                    in += e[v] * dg[v];
                }
            }
            in = row_sum<LPR>(in);
            if (a.norm == FK_GATES_CHOSEN) {
                es = row_sum<LPR>(es);
                const float ginv = es > 0.0f ? 1.0f / es : 0.0f;
                const float inner = in * ginv;
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    const float g = (sel >> v) & 1u ? e[v] * ginv * (dg[v] - inner) : 0.0f;
                    dl[v] = e[v] * inv * (f[v] + shift) + g;
                }
            } else {
                const float inner = in * inv;
#pragma unroll
                for (int v = 0; v < VPL; ++v) dl[v] = e[v] * inv * (f[v] + shift + dg[v] - inner);
            }
        }
        T *out = (T *)a.d_logits + row * a.E + col;
        constexpr int W = 16 / (int)sizeof(T);
        if (a.vec) {
#pragma unroll
            for (int v = 0; v < VPL; v += W) {
                Chunk<T, W> c;
#pragma unroll
                for (int i = 0; i < W; ++i) c.e[i] = (T)dl[v + i];
                if (col + v < a.E) c.store(out + v);
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (col + v < a.E) out[v] = (T)dl[v];
        }
    }
}

int lanes_per_row(int E) {
    int l = 1;
    while (l < 64 && l * 8 < E) l <<= 1;
    return l;
}

template <typename T, bool BWD>
hipError_t dispatch_route(const RouteArgs &a, hipStream_t s) {
    const int lpr = lanes_per_row(a.E);
    const int vpl = a.E > 512 ? 16 : 8;
    const size_t need = (size_t)(kRouteThreads + 2 * a.E + 2) * 4, cols = (size_t)lpr * vpl * 8;
    const size_t lds = need > cols ? need : cols;
    const int64_t per = 256 / lpr;
    const unsigned bgrid = (unsigned)(cdiv(a.T, per) < 4096 ? cdiv(a.T, per) : 4096);
    const unsigned fgrid = (unsigned)route_blocks(a.T, a.E);
#define FK_ROUTE(LPR, VPL)                                                              \
    do {                                                                                \
        if constexpr (BWD) k_route_bwd<T, LPR, VPL><<<bgrid, 256, 0, s>>>(a);           \
        else k_route<T, LPR, VPL><<<fgrid, kRouteThreads, lds, s>>>(a);                 \
    } while (0)
    switch (lpr) {
    case 1: FK_ROUTE(1, 8); break;
    case 2: FK_ROUTE(2, 8); break;
    case 4: FK_ROUTE(4, 8); break;
    case 8: FK_ROUTE(8, 8); break;
    case 16: FK_ROUTE(16, 8); break;
    case 32: FK_ROUTE(32, 8); break;
    default:
        if (vpl == 8) FK_ROUTE(64, 8);
        else FK_ROUTE(64, 16);
    }
#undef FK_ROUTE
    if (!BWD && fgrid > 1) k_route_finish<<<1, kRouteThreads, lds, s>>>(a, (int)fgrid);
    return hipGetLastError();
}

template <bool BWD>
hipError_t dispatch(int dtype, const RouteArgs &a, hipStream_t s) {
    switch (dtype) {
    case FK_F32: return dispatch_route<float, BWD>(a, s);
    case FK_BF16: return dispatch_route<__bf16, BWD>(a, s);
    default: return dispatch_route<_Float16, BWD>(a, s);
    }
}

int chunked(int dtype, const void *logits, const void *out, int64_t ldl, int E) {
    const int v = 16 / (int)dtype_size(dtype);
    return E % v == 0 && ldl % v == 0 && ((uintptr_t)logits & 15) == 0 && ((uintptr_t)out & 15) == 0;
}

}  // namespace

int route_blocks(int64_t T, int E) {
    const int64_t need = cdiv(T > 0 ? T : 1, kRouteThreads / lanes_per_row(E));
    return (int)(need < kRouteMaxBlocks ? need : kRouteMaxBlocks);
}

size_t route_scratch_bytes(int64_t T, int E) { return (size_t)route_blocks(T, E) * (2 * E + 2) * 4; }

hipError_t launch_route(int dtype, const void *logits, int64_t ldl, int64_t T, int E, int k, int norm,
                        const uint8_t *valid, int32_t *ids, float *gates, int32_t *counts, float *losses,
                        int32_t *live, void *scratch, hipStream_t s) {
    RouteArgs a{};
    a.logits = logits, a.ldl = ldl, a.T = T, a.E = E, a.k = k, a.norm = norm, a.valid = valid;
    a.ids = ids, a.gates = gates, a.counts = counts, a.losses = losses, a.live = live, a.part = (float *)scratch;
    a.vec = chunked(dtype, logits, nullptr, ldl, E);
    return dispatch<false>(dtype, a, s);
}

hipError_t launch_route_bwd(int dtype, const void *logits, int64_t ldl, int64_t T, int E, int k, int norm,
                            const uint8_t *valid, const int32_t *ids, const int32_t *counts, const int32_t *live,
                            const float *d_gates, const float *d_losses, void *d_logits, hipStream_t s) {
    RouteArgs a{};
    a.logits = logits, a.ldl = ldl, a.T = T, a.E = E, a.k = k, a.norm = norm, a.valid = valid;
    a.ids_in = ids, a.counts_in = counts, a.live_in = live, a.d_gates = d_gates, a.d_losses = d_losses;
    a.d_logits = d_logits;
    a.vec = chunked(dtype, logits, d_logits, ldl, E);
    return dispatch<true>(dtype, a, s);
}

}  // namespace fk
