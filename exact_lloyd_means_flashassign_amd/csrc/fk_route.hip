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
// A row belongs to a team of 2^m lanes, 8 consecutive experts a lane up to
// E = 512 (16 beyond), so a row's reductions are at most six lane exchanges and
// a lane meets the same experts in every row: the columns' sums stay in its
// registers until the workgroup is done (the counts in LDS, by integer adds,
// whose order does not matter), and leave as one partial row, which a second
// kernel adds in a fixed order (a single workgroup finishes by itself).
//
// The k best: a lane turns its logits into keys (below) and sorts them by a
// network; then the team takes the largest of its lanes' first keys k times,
// the lane that had it moving on to its next.  A key is the logit as a double,
// which leaves 29 bits of its fraction free, with the expert's index in the
// lowest 10, so that one comparison settles ties too and names the expert.
// At many rows this arithmetic, not memory, is the forward pass's bound:
// 262144 rows of 128 experts, k = 8, fp32 take 100 us, the vector units busy for
// 87 % of them, where their bytes alone would take 30; in bf16 96 us.  The
// backward pass, which only reads, scales and writes, takes 62 us (4.7 TB/s; bf16
// 51).  16 rows of 64 experts take 6 us, one launch.  Above 512 experts, 16
// logits a lane, the forward kernel spills 19 to 29 registers.
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
    float *part;  // [blocks][part_row(E)]
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
    return lanes_reduce<LPR>(v, [](float a, float b) { return fmaxf(a, b); });
}

// ---- keys ----
constexpr uint32_t kIndexBits = 1023;  // FK_MAX_EXPERTS - 1
constexpr double kNoKey = -__builtin_inf();

// The larger the logit the larger the key, then the lower the index: the
// index is turned round where a larger fraction makes a larger number.  -inf
// and NaN have no key; +inf stands as 2^128.
__device__ __forceinline__ double key_of(float l, int e) {
    if (!(l > -INFINITY)) return kNoKey;
    const double d = l == INFINITY ? 0x1p128 : (double)(l + 0.0f);  // (-0 is 0)
    uint64_t u = __builtin_bit_cast(uint64_t, d);
    u |= (u >> 63) ? (uint32_t)e : kIndexBits - (uint32_t)e;
    return __builtin_bit_cast(double, u);
}
__device__ __forceinline__ int key_expert(double k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k);
    const uint32_t i = (uint32_t)u & kIndexBits;
    return (int)((u >> 63) ? i : kIndexBits - i);
}
__device__ __forceinline__ float key_logit(double k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k) & ~(uint64_t)kIndexBits;
    return (float)__builtin_bit_cast(double, u);
}

template <int O>
__device__ __forceinline__ double key_neighbour(double k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k);
    const uint64_t r = (uint64_t)neighbour<O>((uint32_t)(u >> 32)) << 32 | neighbour<O>((uint32_t)u);
    return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return __builtin_fmin(a, b); }
template <int LPR, int O = 1>
__device__ __forceinline__ double key_max(double k) {
    if constexpr (O >= LPR) return k;
    else return key_max<LPR, 2 * O>(larger(k, key_neighbour<O>(k)));
}

// Sorts 8 keys, largest first, by a network of 19 comparisons.
__device__ __forceinline__ void sort8(double *k) {
    constexpr int net[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                                {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) {
        const double a = k[net[i][0]], b = k[net[i][1]];
        k[net[i][0]] = larger(a, b);
        k[net[i][1]] = smaller(a, b);
    }
}
// ... and 16, as two sorted eights merged: the larger halves of a and of b
// turned round form a bitonic run each, which three rounds sort.
__device__ __forceinline__ void sort16(double *k) {
    sort8(k);
    sort8(k + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double a = k[i], b = k[15 - i];
        k[i] = larger(a, b);
        k[15 - i] = smaller(a, b);
    }
#pragma unroll
    for (int h = 0; h < 16; h += 8)
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i & o) continue;
                const double a = k[h + i], b = k[h + i + o];
                k[h + i] = larger(a, b);
                k[h + i + o] = smaller(a, b);
            }
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

// A partial row: fp32 sums of p for each expert and of lse^2, up to a multiple
// of four columns; then int32 counts for each expert and live rows, likewise.
__host__ __device__ inline int part_floats(int E) { return (E + 1 + 3) / 4 * 4; }
__host__ __device__ inline int part_row(int E) { return 2 * part_floats(E); }

// The counts, live rows and losses from P partial rows, by one workgroup: 4
// columns a thread, the rows in as many runs as there are threads for, each
// run's loads in flight together.
__device__ __forceinline__ void route_finish(const RouteArgs &a, int P, float *sm) {
    const int E = a.E, F = part_floats(E), chunks = 2 * F / 4;
    const int runs = kRouteThreads / chunks;
    const int c = threadIdx.x % chunks, run = threadIdx.x / chunks;
    float4 f = {0.0f, 0.0f, 0.0f, 0.0f};
    int4 n = {0, 0, 0, 0};
    const float4 *part = reinterpret_cast<const float4 *>(a.part);
    if (run < runs) {
        constexpr int U = 8;
        for (int p0 = run; p0 < P; p0 += U * runs) {
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = p0 + u * runs;
                v[u] = p < P ? part[(size_t)p * chunks + c] : float4{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                f.x += v[u].x, f.y += v[u].y, f.z += v[u].z, f.w += v[u].w;
                n.x += __float_as_int(v[u].x), n.y += __float_as_int(v[u].y);
                n.z += __float_as_int(v[u].z), n.w += __float_as_int(v[u].w);
            }
        }
    }
    // the runs in order; sm: [runs][2 F] and then the totals [2 F]
    float4 *s4 = reinterpret_cast<float4 *>(sm);
    __syncthreads();
    const bool whole = c * 4 >= F;  // integer columns
    if (run < runs)
        s4[run * chunks + c] = whole ? float4{__int_as_float(n.x), __int_as_float(n.y), __int_as_float(n.z), __int_as_float(n.w)} : f;
    __syncthreads();
    float *tot = sm + runs * 2 * F;
    for (int col = threadIdx.x; col < 2 * F; col += kRouteThreads) {
        float t = 0.0f;
        int m = 0;
        for (int r = 0; r < runs; ++r) {
            const float v = sm[r * 2 * F + col];
            t += v;
            m += __float_as_int(v);
        }
        tot[col] = col < F ? t : __int_as_float(m);
        if (col >= F && col < F + E) a.counts[col - F] = m;
        if (col == F + E) a.live[0] = m;
    }
    __syncthreads();
    const int *cnt = reinterpret_cast<const int *>(tot) + F;
    // all slots, and sum_e counts_e psum_e
    float all = 0.0f, bal = 0.0f;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
        all += (float)cnt[e];
        bal += (float)cnt[e] * tot[e];
    }
    all = lanes_sum<64>(all);
    bal = lanes_sum<64>(bal);
    __shared__ float s_all[kRouteThreads / 64], s_bal[kRouteThreads / 64];
    if ((threadIdx.x & 63) == 0) {
        s_all[threadIdx.x >> 6] = all;
        s_bal[threadIdx.x >> 6] = bal;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.0f, b = 0.0f;
        for (int w = 0; w < kRouteThreads / 64; ++w) {
            t += s_all[w];
            b += s_bal[w];
        }
        const float live = (float)(cnt[E] > 0 ? cnt[E] : 1);
        a.losses[0] = (float)E * (b / (t > 0.0f ? t : 1.0f)) / live;
        a.losses[1] = tot[E] / live;
    }
}

template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a) {
    constexpr int RPB = kRouteThreads / LPR;  // rows a round
    constexpr int COLS = LPR * VPL;
    extern __shared__ __attribute__((aligned(16))) float sm[];
    const int lane = threadIdx.x % LPR;
    const int col = lane * VPL;
    int *counts = reinterpret_cast<int *>(sm) + kRouteThreads / 64 * COLS;
    for (int i = threadIdx.x; i < COLS; i += kRouteThreads) counts[i] = 0;
    __syncthreads();
    float psum[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) psum[v] = 0.0f;
    float zsum = 0.0f;
    int nlive = 0;
    const int64_t step = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    // the next row's logits are sent for before this one is worked on: in fp32
    // they are under way meanwhile (the row's valid flag, if there are any, is
    // waited for first); 16-bit ones are converted, and so waited for, at once
    float ahead[VPL];
    auto fetch = [&](int64_t r) {
        load_row<T, VPL>(a, r, col, r < a.T && (a.valid == nullptr || a.valid[r] != 0), ahead);
    };
    fetch(row);
    for (; row < a.T; row += step) {
        float l[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) l[v] = ahead[v];
        fetch(row + step);
        float m = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            m = fmaxf(m, l[v]);  // the larger of the two, NaN ignored
            nan = nan || l[v] != l[v];
        }
        m = row_max<LPR>(m);
        const float nans = row_sum<LPR>(nan ? 1.0f : 0.0f);
        int32_t *ids = a.ids + row * a.k;
        float *gates = a.gates + row * a.k;
        if (m == -INFINITY && nans == 0.0f) {
            for (int j = lane; j < a.k; j += LPR) {
                ids[j] = a.E;
                gates[j] = 0.0f;
            }
            continue;
        }
        float e[VPL], s = 0.0f;
        double key[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            e[v] = exp_neg(l[v] - m);
            s += e[v];
            key[v] = key_of(l[v], col + v);
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
        if constexpr (VPL == 8) sort8(key);
        else sort16(key);
        // Lane j % LPR of the team keeps choice j and looks at it once LPR of
        // them are made (gates are written before their scale is known if
        // there are more, and scaled by the lane that wrote them).
        float gsum = 0.0f, mine = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += LPR) {
            const int jn = a.k - j0 < LPR ? a.k - j0 : LPR;
            double chosen = kNoKey;
            for (int j = 0; j < jn; ++j) {
                const double best = key_max<LPR>(key[0]);
                chosen = lane == j ? best : chosen;
                if (key[0] == best) {  // keys differ: the lane that had it (or none is left)
#pragma unroll
                    for (int v = 0; v + 1 < VPL; ++v) key[v] = key[v + 1];
                    key[VPL - 1] = kNoKey;
                }
            }
            const bool any = chosen != kNoKey;
            const int at = any ? key_expert(chosen) : a.E;
            mine = any ? exp_neg(key_logit(chosen) - m) : 0.0f;
            gsum += row_sum<LPR>(mine);
            if (any) atomicAdd(&counts[at], 1);
            if (lane < jn) {
                ids[j0 + lane] = at;
                if (a.k > LPR) gates[j0 + lane] = mine;
            }
        }
        const float scale = a.norm == FK_GATES_CHOSEN ? 1.0f / gsum : inv;
        for (int j = lane; j < a.k; j += LPR) {
            const float g = a.k > LPR ? gates[j] : mine;
            gates[j] = g == 0.0f ? 0.0f : g * scale;
        }
    }
    // the teams' columns: lanes of a wave that own the same experts, then the
    // waves in order through LDS
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
#pragma unroll
        for (int o = LPR; o < 64; o <<= 1) psum[v] += __shfl_xor(psum[v], o, 64);
    }
    zsum = lanes_sum<64>(zsum);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) nlive += __shfl_xor(nlive, o, 64);
    constexpr int WV = kRouteThreads / 64;
    const int wv = threadIdx.x >> 6;
    __shared__ float s_z[WV];
    __shared__ int s_live[WV];
    // sm: each wave's sums, then the counts
    if ((threadIdx.x & 63) < LPR) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) sm[wv * COLS + col + v] = psum[v];
    }
    if ((threadIdx.x & 63) == 0) {
        s_z[wv] = zsum;
        s_live[wv] = nlive;
    }
    __syncthreads();
    const int F = part_floats(a.E);
    float *out = a.part + (size_t)blockIdx.x * 2 * F;
    for (int c = threadIdx.x; c < F; c += kRouteThreads) {
        float z = 0.0f;
        int n = 0;
        if (c < a.E) {
#pragma unroll
            for (int w = 0; w < WV; ++w) z += sm[w * COLS + c];
        } else if (c == a.E) {
            for (int w = 0; w < WV; ++w) {
                z += s_z[w];
                n += s_live[w];
            }
        }
        out[c] = z;
        out[F + c] = __int_as_float(c < a.E ? counts[c] : n);
    }
    if (gridDim.x == 1) {
        __syncthreads();  // the partial row is read back by the same workgroup
        route_finish(a, 1, sm);
    }
}

__global__ __launch_bounds__(kRouteThreads) void k_route_finish(RouteArgs a, int P) {
    extern __shared__ __attribute__((aligned(16))) float sm[];
    route_finish(a, P, sm);
}

// A lane j % LPR of the team takes choice j: it reads that logit again, the
// team sums what the gates' softmax needs, and the choices' parts reach the
// lanes that own the experts through LDS.
template <typename T, int LPR, int VPL>
__global__ __launch_bounds__(256) void k_route_bwd(RouteArgs a) {
    constexpr int RPB = 256 / LPR;
    __shared__ __attribute__((aligned(16))) float parts[256 * VPL];
    const int lane = threadIdx.x % LPR;
    const int col = lane * VPL;
    float *own = parts + threadIdx.x * VPL, *team = own - col;
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
            float shift = -pv * inv;
            if (dz != 0.0f) shift += dz * 2.0f * (m + logf(s)) / n;
            if (a.d_gates != nullptr) {
                const int32_t *ids = a.ids_in + row * a.k;
                const float *dg = a.d_gates + row * a.k;
                const T *again = (const T *)a.logits + row * a.ldl;
                float es = 0.0f, in = 0.0f;
                for (int j = lane; j < a.k; j += LPR) {
                    const int id = ids[j];
                    if ((unsigned)id >= (unsigned)a.E) continue;
                    const float ej = exp_neg((float)again[id] - m);
                    es += ej;
                    in += ej * dg[j];
                }
                es = row_sum<LPR>(es);
                in = row_sum<LPR>(in);
                const bool chosen = a.norm == FK_GATES_CHOSEN;
                const float scale = chosen ? (es > 0.0f ? 1.0f / es : 0.0f) : inv;
                const float inner = in * scale;
#pragma unroll
                for (int v = 0; v < VPL; ++v) own[v] = 0.0f;
                // (the team's lanes are in one wave: their LDS accesses are in order)
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                for (int j = lane; j < a.k; j += LPR) {
                    const int id = ids[j];
                    if ((unsigned)id >= (unsigned)a.E) continue;
                    const float g = exp_neg((float)again[id] - m) * scale;
                    team[id] = chosen ? g * (dg[j] - inner) : g * dg[j];
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int v = 0; v < VPL; ++v) dl[v] = own[v];
                if (!chosen) shift -= inner;
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v) dl[v] += e[v] * inv * (f[v] + shift);
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
    // the waves' sums and the counts of every column; the finish's runs and totals
    const int row = part_row(a.E), runs = kRouteThreads / (row / 4);
    const size_t need = (size_t)(runs + 1) * row * 4, cols = (size_t)lpr * vpl * 4 * (kRouteThreads / 64 + 1);
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

size_t route_scratch_bytes(int64_t T, int E) { return (size_t)route_blocks(T, E) * part_row(E) * 4; }

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
