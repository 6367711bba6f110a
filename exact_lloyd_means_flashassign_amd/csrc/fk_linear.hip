// Products with an epilogue for gfx950, and their gradients, for one weight
// matrix or one per group of rows.
//
//   z[p] = X[row(p)] W_g^T + b_g,   Y[slot(p)] = act(z[p]) + R[slot(p)]
//   dZ = dY act'(z),   dX[slot(p)] = dZ[p] W_g,   dW_g = sum_p dZ[p]^T X[row(p)],   db_g = sum_p dZ[p]
//
// p runs over the positions of a slot list sorted by group: slot(p) =
// slots[p], row(p) = slots[p] / share, and group g owns [offsets[g],
// offsets[g+1]).  A plain product has one group and slot(p) = row(p) = p.
//
// Sums are fp32 in the matrix instructions' accumulators; bias, activation and
// residual are applied to them, and each output is rounded once.  dZ is
// rounded to the operands' type before it is multiplied, as the 16-bit matrix
// instructions need; db is the sum of the unrounded values.  Three kernels
// share the work: tiles (k_product), which are bound by the matrix units; a few
// rows (k_product_few), bound by the stream of the weights; and the
// element-wise step of the gradients (k_act_grad), bound by memory.
#include <type_traits>

#include "fk.h"
#include "fk_block.h"
#include "fk_internal.h"
#include "fk_rows.h"

namespace fk {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void *lds_ptr;
typedef const __attribute__((address_space(1))) void *glb_ptr;

// 16 bytes of zeros: what a lane reads in the place of elements past the end
// of the sum, so that every lane's load stays in bounds.
__device__ __attribute__((aligned(16))) const uint32_t g_zeros[4] = {0, 0, 0, 0};

// A lane's 16 bytes of an operand for one 32-byte step of the sum, and the
// products on them: both operands hold the same elements of the sum at the
// same places, whichever they are.
template <typename T>
struct Mma;
template <>
struct Mma<__bf16> {
    typedef v8bf Frag;
    static __device__ __forceinline__ v16f m32(Frag a, Frag b, v16f c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ v4f m16(Frag a, Frag b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mma<_Float16> {
    typedef v8h Frag;
    static __device__ __forceinline__ v16f m32(Frag a, Frag b, v16f c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ v4f m16(Frag a, Frag b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mma<float> {
    typedef v4f Frag;
    static __device__ __forceinline__ v16f m32(Frag a, Frag b, v16f c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ v4f m16(Frag a, Frag b, v4f c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// ---- activations ----------------------------------------------------------------
//
// In two forms, each to the accuracy of what it is for.  FINE, for results that
// leave in fp32: the mathematical library's exponential and complementary error
// function and a correctly rounded quotient, a few ulp of the result, small
// results too.  Otherwise, for results that are rounded to 16 bits: the
// hardware's exponential and reciprocal and an approximation of erf, good to
// 1.5e-7 of |z| where the rounding alone takes 4.9e-4 (fp16) or more of the
// result.  In fp32, 16384 x 4096 by a sum of 128, the one takes 244 us with gelu
// and 219 with silu, the other 218 and 198, no activation 184.

// 2^x and 1/x by the hardware's instructions (about an ulp each); an infinite
// 2^x gives a logistic of 0.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
template <bool FINE>
__device__ __forceinline__ float logistic(float x) {
    if constexpr (FINE) return 1.0f / (1.0f + expf(-x));
    else return __builtin_amdgcn_rcpf(1.0f + exp_of(-x));
}

// (1 + erf(z / sqrt 2)) / 2, and e^(-z^2/2).  The fast form by the rational
// approximation 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical
// Functions (1964), whose error is below 1.5e-7 in erf and which needs the
// exponential anyway.
template <bool FINE>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    if constexpr (FINE) {
        e = expf(-0.5f * z * z);
        return 0.5f * erfcf(-0.707106781f * z);
    }
    const float x = fabsf(z) * 0.707106781f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
    float p = 1.061405429f;
    p = __builtin_fmaf(p, t, -1.453152027f);
    p = __builtin_fmaf(p, t, 1.421413741f);
    p = __builtin_fmaf(p, t, -0.284496736f);
    p = __builtin_fmaf(p, t, 0.254829592f);
    e = exp_of(-0.5f * z * z);
    const float tail = 0.5f * p * t * e;  // the smaller of the two sides
    return z < 0.0f ? tail : 1.0f - tail;
}

// twice the argument of gelu_tanh's tanh: z (1 + tanh u) / 2 = z logistic(2 u)
__device__ __forceinline__ float tanh_arg(float z) { return 1.59576912f * (z + 0.044715f * z * z * z); }

// the activation of N values (the choice outside their loop)
template <bool FINE, int N>
__device__ __forceinline__ void activate(int act, float (&z)[N]) {
    if (act == FK_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];
    } else if (act == FK_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e;
            z[i] *= normal_cdf<FINE>(z[i], e);
        }
    } else if (act == FK_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= logistic<FINE>(tanh_arg(z[i]));
    } else if (act == FK_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= logistic<FINE>(z[i]);
    }
}

// d[i] *= the activation's slope at z[i].  Where the slope has come to its
// limit (0 or 1), z is held back so that its powers stay finite.
template <bool FINE, int N>
__device__ __forceinline__ void times_slope(int act, const float (&z)[N], float (&d)[N]) {
    if (act == FK_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] *= z[i] > 0.0f ? 1.0f : 0.0f;
    } else if (act == FK_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float c = z[i] != z[i] ? z[i] : fminf(fmaxf(z[i], -64.0f), 64.0f);
            float e;
            const float s = normal_cdf<FINE>(c, e);
            d[i] *= s + c * e * 0.398942280f;
        }
    } else if (act == FK_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float c = z[i] != z[i] ? z[i] : fminf(fmaxf(z[i], -64.0f), 64.0f);
            const float s = logistic<FINE>(tanh_arg(c));
            d[i] *= s + c * s * (1.0f - s) * 1.59576912f * (1.0f + 0.134145f * c * c);
        }
    } else if (act == FK_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float c = z[i] != z[i] ? z[i] : fminf(fmaxf(z[i], -128.0f), 128.0f);
            const float s = logistic<FINE>(c);
            d[i] *= s * (1.0f + c * (1.0f - s));
        }
    }
}

// ---- rows and groups --------------------------------------------------------------

// Where position p lies in a matrix: p itself, or slots[p] / div (a slot out
// of range is taken as the last one, so that no list can reach past the
// matrix).
struct RowMap {
    const int32_t *slots;
    int32_t last;        // the largest slot
    uint32_t mul, shift;  // s / div = (mulhi(s, mul) + s) >> shift for s < 2^31
    __device__ __forceinline__ int64_t operator()(int64_t p) const {
        if (slots == nullptr) return p;
        return of(slots[p]);
    }
    __device__ __forceinline__ int64_t of(int32_t s) const {
        const uint32_t u = (uint32_t)s < (uint32_t)last ? (uint32_t)s : (uint32_t)last;
        return (__umulhi(u, mul) + u) >> shift;
    }
};

RowMap row_map(const int32_t *slots, int64_t M, int div) {
    RowMap r{slots, (int32_t)(M - 1), 0, 0};
    while (((int64_t)1 << r.shift) < div) ++r.shift;
    r.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << r.shift) - (uint64_t)div)) / (uint64_t)div + 1);
    return r;
}

// offsets[g] held inside [0, M], rising or not as the caller gave it
__device__ __forceinline__ int64_t group_at(const int32_t *offsets, int g, int64_t M) {
    const int32_t o = offsets[g];
    return o < 0 ? 0 : ((int64_t)o < M ? (int64_t)o : M);
}

// a value that is the same in every lane, as a scalar
__device__ __forceinline__ int64_t scalar(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Finds row tile `want` among the groups' tiles of `rows` rows (groups of
// `skip` rows or fewer have none).  Group G stands for the positions past the
// last group (with_rest).  Every lane of a wave calls it and gets the same
// answer.  Returns the number of tiles in all; g = -1 if there is no such tile.
struct TileAt {
    int g;
    int64_t p0, p1;  // its positions
};
__device__ __forceinline__ int64_t find_tile(const int32_t *offsets, int G, int64_t M, int rows, int skip,
                                             bool with_rest, int64_t want, TileAt &t) {
    t.g = -1;
    t.p0 = t.p1 = 0;
    const int lane = threadIdx.x & 63;
    const int n = G + (with_rest ? 1 : 0);
    int64_t before = 0;
    for (int g0 = 0; g0 < n; g0 += 64) {
        const int g = g0 + lane;
        int64_t a = 0, b = 0;
        if (g < n) {
            a = group_at(offsets, g, M);
            b = g < G ? group_at(offsets, g + 1, M) : M;
        }
        const int64_t cnt = b > a ? b - a : 0;
        const int tiles = g < G && cnt <= skip ? 0 : (int)((cnt + rows - 1) / rows);
        int inc = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(inc, o, 64);
            if (lane >= o) inc += up;
        }
        const int64_t mine = before + inc - tiles;
        const uint64_t hit = __ballot(want >= mine && want < mine + tiles);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int64_t first = __shfl(mine, src, 64);
            const int64_t ga = __shfl(a, src, 64), gb = __shfl(b, src, 64);
            t.g = g0 + src;
            t.p0 = ga + (want - first) * rows;
            t.p1 = t.p0 + rows < gb ? t.p0 + rows : gb;
        }
        before += __shfl(inc, 63, 64);
    }
    return before;
}

// This workgroup among those of a long grid.  A dimension of a launch takes fewer
// than 2^32 threads, 2^24 workgroups of 256; where a matrix of one column has
// more tiles than that, the grid goes on in z.  Workgroups past its end find no
// tile.
constexpr int kGridBits = 23;
__device__ __forceinline__ int64_t workgroup() { return (int64_t)blockIdx.z << kGridBits | blockIdx.x; }
inline dim3 long_grid(int64_t n, int y = 1) {
    if (n >> kGridBits == 0) return dim3((unsigned)n, (unsigned)y);
    return dim3(1u << kGridBits, (unsigned)y, (unsigned)cdiv(n, (int64_t)1 << kGridBits));
}

// The tile of this workgroup when `total` of them are spread over the 8 XCDs,
// which take workgroups in turn: each XCD gets a run of consecutive tiles, so
// that the tiles that share operands share an L2.  -1: none.
__device__ __forceinline__ int64_t xcd_tile(int64_t id, int64_t total) {
    const int64_t x = id & 7, i = id >> 3, q = total >> 3, r = total & 7;
    if (i >= q + (x < r ? 1 : 0)) return -1;
    return x * q + (x < r ? x : r) + i;
}

// ---- the tiled product -------------------------------------------------------------

enum { kFwd = 0, kDx = 1, kDw = 2 };

struct LinArgs {
    const void *A, *B;
    void *C, *Z;
    const void *bias, *R;
    float *part;  // split sums: [splits][rows of C in position order][N]
    const int32_t *offsets;
    RowMap amap, bmap, cmap;
    int64_t lda, ldb, ldc, ldz, ldr;
    int64_t gsb, gsc, gsbias;  // group strides of B, C, bias
    int64_t M;                 // positions
    int64_t rows, N;           // rows (of a group for kDw) and columns of C
    int64_t ka, kb;            // where the sum ends in A and in B
    int G, act, splits, skip, cf32, bf32;
    int chunked;               // C, R and Z can be written and read by whole chunks of 8 columns
};

typedef const __attribute__((address_space(3))) void *lds_at;

// 16 bytes a lane from memory to LDS, lane after lane from `lds` (the same in
// every lane).  Written in assembly because the compiler, which cannot tell
// that a transposing read and a load under way touch different tiles, would
// wait for every load before the next such read; here the caller waits
// (vmcnt) before it reads what was loaded.  No register is written, and the
// address is taken when the instruction issues.  m0, which holds the place in
// LDS, needs a wait state before the load.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is never live across statements
// from a scalar base and a lane's offset in bytes (no address arithmetic in
// the lanes: 1251 TFLOP/s where lane addresses gave 1210, 16384 x 8192 x 4096)
__device__ __forceinline__ void load_to_lds(const void *base, uint32_t off, lds_at lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %2" ::"v"(off), "s"(at),
                 "s"((glb_ptr)base)
                 : "m0");
}
// from a lane's address
__device__ __forceinline__ void load_to_lds(const void *src, lds_at lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"((glb_ptr)src), "s"(at)
                 : "m0");
}
// 4 bytes a lane
__device__ __forceinline__ void dword_to_lds(const void *src, lds_at lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"((glb_ptr)src), "s"(at) : "m0");
}
#pragma clang diagnostic pop

constexpr int kTileThreads = 256;  // 4 waves, one a SIMD

// One operand's tile: BS rows (or columns) of C by 128 bytes of the sum, as
// two parts of BS / 2 rows (columns) in LDS, each of 16-byte chunks.
//   KM (the sum is contiguous in memory): LDS row r holds 8 chunks, chunk c at
//     place c ^ (r >> 1 & 7): 16 lanes that read the same chunk of 16
//     consecutive rows meet 16 different places of the 64 banks.
//   otherwise (rows of the operand are steps of the sum): LDS row k holds the
//     part's columns, chunk c at place c ^ mn_turn(k): the four rows that a
//     transposing read takes lie on different banks.
// Loads go from memory straight to LDS, 16 bytes a lane, each lane fetching
// the chunk that belongs at its place; 8 lanes take the whole 128 bytes of a
// row, so that every request to L2 is a full line.
template <typename T, bool KM, int BS>
struct Operand {
    typedef const __attribute__((address_space(3))) T *Lds;
    static constexpr int NT = kTileThreads;
    static constexpr int E = 16 / (int)sizeof(T);       // elements a chunk
    static constexpr int BK = 8 * E;                    // steps of the sum in a tile
    static constexpr int PR = BS / 2;                   // rows (columns) of a part
    static constexpr int PART = PR * BK;                // elements of a part
    static constexpr int IT = PR * 8 / NT;              // loads a thread for a part
    static constexpr int CPR = KM ? 8 : PR / E;         // chunks a LDS row
    static constexpr int STEP = NT / CPR;               // LDS rows a load of all threads covers
    const char *base;               // (scalar) what the offsets of the split's first tile count from
    int64_t adv;                    // (scalar) bytes from one tile to the next
    uint32_t off[KM ? 2 * IT : IT];  // the lane's chunks, in bytes
    int over;                       // not KM: bytes from the first part's columns to the second's
    int kofs;                       // KM: this thread's chunk in the 128 bytes; else its row of the sum
    uint32_t pitch, col;            // not KM: bytes of a row, and the lane's columns in it
    RowMap map;
    int64_t pos0;

    static __device__ __forceinline__ int mn_turn(int k) { return CPR >= 16 ? (k & 3) << 2 : ((k >> 1) & 1) << 2; }

    // KM: rows [r0, r0 + n) of C at positions; out of range rows repeat the last
    __device__ __forceinline__ void init_km(const T *m0, int64_t ld, const RowMap &m, int64_t r0, int64_t n,
                                            int64_t k0) {
        const int row = threadIdx.x >> 3;
        kofs = ((threadIdx.x & 7) ^ ((row >> 1) & 7)) * E;
        adv = BK * sizeof(T);
        const bool mapped = m.slots != nullptr;
        base = (const char *)(m0 + (mapped ? 0 : r0 * ld) + k0);
#pragma unroll
        for (int i = 0; i < 2 * IT; ++i) {
            const int64_t r = row + i * STEP < n ? row + i * STEP : n - 1;
            off[i] = (uint32_t)(((mapped ? m(r0 + r) : r) * ld + kofs) * (int64_t)sizeof(T));
        }
    }
    // not KM: columns [c0, cols), the sum over positions from pos; out of range
    // columns repeat the last chunk
    __device__ __forceinline__ void init_mn(const T *m0, int64_t ld, const RowMap &m, int64_t c0, int64_t cols,
                                            int64_t pos, int64_t k0) {
        kofs = threadIdx.x / CPR;
        const int64_t c = c0 + (int64_t)((threadIdx.x % CPR) ^ mn_turn(kofs)) * E;
        const int64_t lastc = (cols - 1) / E * E;
        const int64_t first = c < lastc ? c : lastc, second = c + PR < lastc ? c + PR : lastc;
        over = (int)(second - first) * (int)sizeof(T);
        col = (uint32_t)(first * sizeof(T));
        pitch = (uint32_t)(ld * sizeof(T));
        map = m;
        pos0 = pos;
        const bool mapped = m.slots != nullptr;
        adv = mapped ? 0 : BK * ld * (int64_t)sizeof(T);
        base = (const char *)(m0 + (mapped ? 0 : (pos + k0) * ld));
#pragma unroll
        for (int i = 0; i < IT; ++i) off[i] = (uint32_t)(kofs + i * STEP) * pitch + col;
    }
    // not KM, rows by slots: a wave keeps the slots of four tiles in LDS, 64
    // places each.  A tile's slots are sent for four tiles ahead (send_rows),
    // read three ahead (read_rows) and turned into the offsets of the loads
    // (take_rows) when these are due.  A scalar load instead would make every
    // LDS read of the wave wait for it, a vector load would wait for all loads
    // to LDS under way.
    typedef const __attribute__((address_space(3))) int32_t *Ring;
    static constexpr int kRing = 4 * 64;
    Ring ring;
    int32_t slot[KM ? 1 : IT];
    // (kend > 0: where the sum ends)
    __device__ __forceinline__ void send_rows(int64_t tile, int64_t k0, int64_t kend) const {
        if constexpr (!KM) {
            if (map.slots != nullptr) {
                const int64_t k = k0 + (threadIdx.x & 63);
                dword_to_lds(map.slots + pos0 + (k < kend ? k : kend - 1), ring + (tile & 3) * 64);
            }
        }
    }
    __device__ __forceinline__ void read_rows(int64_t tile) {
        if constexpr (!KM) {
            if (map.slots != nullptr) {
#pragma unroll
                for (int i = 0; i < IT; ++i) slot[i] = ring[(tile & 3) * 64 + kofs + i * STEP];
            }
        }
    }
    __device__ __forceinline__ void take_rows() {
        if constexpr (!KM) {
            if (map.slots != nullptr) {
#pragma unroll
                for (int i = 0; i < IT; ++i) off[i] = (uint32_t)map.of(slot[i]) * pitch + col;
            }
        }
    }
    // Load i of a part of tile `tile`, every step of which is in the sum
    __device__ __forceinline__ void issue(const char *from, Lds part, int wave, int half, int i) const {
        const uint32_t o = KM ? off[half * IT + i] : off[i] + (half ? over : 0);
        load_to_lds(from, o, part + (i * NT + wave * 64) * E);
    }
    // the same where only `rem` steps of it are left: zeros past them
    __device__ __forceinline__ void issue_end(const char *from, Lds part, int wave, int half, int i, int rem) const {
        const uint32_t o = KM ? off[half * IT + i] : off[i] + (half ? over : 0);
        const int k = KM ? kofs : kofs + i * STEP;
        load_to_lds(k < rem ? (const void *)(from + o) : (const void *)g_zeros, part + (i * NT + wave * 64) * E);
    }
    // The lane's 16 bytes for rows (columns) [r0, r0 + 32) of a part and
    // 32-byte step s
    __device__ __forceinline__ static typename Mma<T>::Frag frag(Lds lds, int r0, int s) {
        const int lane = threadIdx.x & 63, l = lane & 31, h = lane >> 5;
        if constexpr (KM) {
            const int r = r0 + l;
            typedef const __attribute__((address_space(3))) typename Mma<T>::Frag *P;
            return *(P)(lds + (r * 8 + ((s * 2 + h) ^ ((r >> 1) & 7))) * E);
        } else if constexpr (sizeof(T) == 4) {
            typename Mma<T>::Frag f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = s * 8 + h * 4 + i, c = r0 + l;
                f[i] = lds[k * PR + ((c / E) ^ mn_turn(k)) * E + c % E];
            }
            return f;
        } else {
            // groups of 16 lanes read 4 rows of 16 columns and get a column
            // (4 steps of the sum) each
            const int i = lane & 15, c = r0 + ((lane >> 4) & 1) * 16 + (i & 3) * 4;
            const int k = s * 16 + h * 8 + (i >> 2);
            const Lds q = lds + k * PR + ((c / E) ^ mn_turn(k)) * E + c % E;
            typedef __attribute__((address_space(3))) v4s *P;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)q);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(q + 4 * PR));
            const v8s both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(typename Mma<T>::Frag, both);
        }
    }
};

// Eight neighbouring values of a row of C through the epilogue and out.
template <typename T>
struct Epilogue {
    float bias[8];
    int64_t col;
    int n;  // columns of the eight that exist
    __device__ __forceinline__ void init(const LinArgs &a, int g, int64_t c) {
        col = c;
        const int64_t left = a.N - c;
        n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bias[i] = 0.0f;
            if (a.bias != nullptr && i < n) {
                const int64_t at = (int64_t)g * a.gsbias + c + i;
                bias[i] = a.bf32 ? ((const float *)a.bias)[at] : (float)((const T *)a.bias)[at];
            }
        }
    }
    // SURE: all eight exist, on whole chunks
    template <bool SURE = false>
    static __device__ __forceinline__ void put(T *q, const float (&v)[8], int n) {
        constexpr int E = 16 / (int)sizeof(T);
        if (SURE || (n == 8 && ((uintptr_t)q & 15) == 0)) {
#pragma unroll
            for (int j = 0; j < 8; j += E) {
                Chunk<T, E> o;
#pragma unroll
                for (int i = 0; i < E; ++i) o.e[i] = (T)v[j + i];
                o.store(q + j);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) q[i] = (T)v[i];
        }
    }
    template <bool SURE = false>
    static __device__ __forceinline__ void get(const T *q, float (&v)[8], int n) {
        constexpr int E = 16 / (int)sizeof(T);
        if (SURE || (n == 8 && ((uintptr_t)q & 15) == 0)) {
#pragma unroll
            for (int j = 0; j < 8; j += E) {
                Chunk<T, E> o;
                o.load(q + j);
#pragma unroll
                for (int i = 0; i < E; ++i) v[j + i] = (float)o.e[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)q[i] : 0.0f;
        }
    }
    // zeros in row crow of C, and of the pre-activations
    __device__ __forceinline__ void zero(const LinArgs &a, int64_t crow) const {
        const float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (a.cf32) Epilogue<float>::put((float *)a.C + crow * a.ldc + col, v, n);
        else put((T *)a.C + crow * a.ldc + col, v, n);
        if (a.Z != nullptr) put((T *)a.Z + crow * a.ldz + col, v, n);
    }
    // N rows of C, eight columns of each; crow: the row (kDw: within its
    // group), below 0: none.  SURE: every row and column exists, on whole chunks.
    // SURE comes with the residual's chunks, which were sent for earlier.
    struct Eight {
        static constexpr int E = 16 / (int)sizeof(T);
        Chunk<T, E> c[8 / E];
        __device__ __forceinline__ void load(const T *p) {
#pragma unroll
            for (int i = 0; i < 8 / E; ++i) c[i].load(p + i * E);
        }
        __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (float)c[i / E].e[i % E];
        }
    };
    // GRAD: a gradient's product, which has no bias, activation or residual.
    template <bool SURE, bool GRAD, int N>
    __device__ __forceinline__ void out(const LinArgs &a, int g, const int64_t (&crow)[N], float (&v)[N * 8],
                                        const Eight *res) const {
        if (!SURE && n == 0) return;
        if constexpr (!GRAD) finish<SURE>(a, crow, v, res);
        const int64_t first = (int64_t)g * a.gsc + col;
        if (sizeof(T) != 4 && a.cf32) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (SURE || crow[k] >= 0)
                    Epilogue<float>::template put<SURE>((float *)a.C + first + crow[k] * a.ldc, *(const float(*)[8])(v + k * 8), n);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (SURE || crow[k] >= 0)
                    put<SURE>((T *)a.C + first + crow[k] * a.ldc, *(const float(*)[8])(v + k * 8), n);
        }
    }
    template <bool SURE, int N>
    __device__ __forceinline__ void finish(const LinArgs &a, const int64_t (&crow)[N], float (&v)[N * 8],
                                           const Eight *res) const {
        float r[N][8];
        if (a.R != nullptr) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (SURE) {
                    res[k].values(r[k]);
                } else if (crow[k] >= 0) {
                    get((const T *)a.R + crow[k] * a.ldr + col, r[k], n);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k * 8 + i] += bias[i];
        if (a.Z != nullptr) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (SURE || crow[k] >= 0)
                    put<SURE>((T *)a.Z + crow[k] * a.ldz + col, *(const float(*)[8])(v + k * 8), n);
        }
        if (sizeof(T) == 4 || a.cf32) activate<true>(a.act, v);
        else activate<false>(a.act, v);
        if (a.R != nullptr) {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k * 8 + i] += r[k][i];
        }
    }
};

// BS x BS of C a workgroup of 2 x 2 waves, the sum in tiles of 128 bytes of
// each row, two tiles of both operands in LDS.
//
// Bound by the matrix units: a wave's products take 2048 cycles a tile (BS =
// 256), and everything else is sent between them.  Each operand's tile lies in
// two parts, and a wave's block of C takes rows from both parts of A and
// columns from both parts of B, so a tile is four quarters: A0 B0, A0 B1,
// A1 B1, A1 B0.  While one quarter is multiplied from registers, the part
// that the next one lacks is read, and after every two quarters, once all
// waves have two parts in registers (a barrier), these parts' places are
// refilled with the tile after the next, four parts ahead of use: loads are
// spread evenly over the products and have most of two tiles' time to arrive.
// One wave a SIMD holds 128 x 128 of C in 256 accumulation registers: 8 waves
// of 128 x 64 read 1.5 times as much from LDS.
//
// Measured in bf16 at 16384 x 8192 x 4096: forward 780 to 810 us (1360 to 1410
// TFLOP/s), dX 815, dW 780 to 795, where the library's product takes 743
// (1480); with gelu and a residual in the epilogue the forward pass takes 950 to
// 1030.  Over the whole kernel the matrix units are busy 60 % of the time there,
// 65 % in dX and 75 % in dW of 16384 x 4096 x 4096, at the 1.55 to 1.63 GHz that
// the card then sustains; the rest is the loads' issue between the products and a
// workgroup's first loads and last stores, which nothing overlaps with one
// workgroup a CU.  The gradients' tiles of 256 spill 2 and 6 registers, outside
// the loop.  In fp32 tiles of 128 reach 140 to 147 TFLOP/s (8192 x 8192 x 2048
// forward 1876 to 1974 us, the library 1852), and 61 to 67 where a few are left
// for a second round (5003 x 1001 x 769, silu and residual: 320 tiles on 256 CUs,
// 115 to 126 us, and 10 for laying out rows of 769).
template <typename T, int KIND, int BS>
__global__ __launch_bounds__(kTileThreads)
__attribute__((amdgpu_waves_per_eu(BS == 256 ? 1 : 2, BS == 256 ? 1 : 2))) void k_product(LinArgs a, int64_t mtiles,
                                                                                          int64_t ntiles) {
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int BK = 8 * E;
    constexpr int BM = BS, BN = BS;
    constexpr int TB = BS / 128;  // 32-row (column) blocks of a part that a wave takes
    constexpr bool AKM = KIND != kDw, BKM = KIND == kFwd;
    constexpr bool SPLITS = BS == 128;  // sums are split where there are few tiles: never large ones
    typedef Operand<T, AKM, BS> OpA;
    typedef Operand<T, BKM, BS> OpB;
    constexpr int PART = OpA::PART, IT = OpA::IT;
    static_assert(OpA::PART == OpB::PART && OpA::IT == OpB::IT, "parts of one size");
    // A0, A1 of even tiles, A0, A1 of odd ones, then B's
    __shared__ __attribute__((aligned(256))) T smem[8 * PART];
    __shared__ __attribute__((aligned(256))) int32_t rings[KIND == kDw ? 4 * 2 * OpA::kRing : 1];
    typedef const __attribute__((address_space(3))) T *Lds;
    const Lds parts = (Lds)smem;

    // ---- which tile ----
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.y;
    TileAt t{0, 0, 0};
    int64_t nt, r0, nrows;   // column tile; first row of C and rows of it in the tile
    int64_t kbeg = 0, ka = a.ka, kb = a.kb;
    int64_t pos = 0;         // kDw: the group's first position
    if constexpr (KIND == kDw) {
        // every XCD takes a run of every group's tiles: groups differ in the
        // length of their sums, so runs of whole groups would not be even
        const int64_t per = mtiles * ntiles, run = (per + 7) >> 3;
        const int64_t id = workgroup(), i = id >> 3;
        t.g = (int)(i / run);
        const int64_t in = (id & 7) * run + i % run;
        if (in >= per || t.g >= a.G) return;
        nt = in % ntiles;
        r0 = in / ntiles * BM;
        nrows = a.rows - r0 < BM ? a.rows - r0 : BM;
        int64_t p1 = a.M;
        if (a.offsets != nullptr) {
            pos = group_at(a.offsets, t.g, a.M);
            p1 = group_at(a.offsets, t.g + 1, a.M);
        }
        ka = kb = p1 > pos ? p1 - pos : 0;
    } else if (a.offsets == nullptr) {
        // runs of 8 row tiles by all column tiles
        const int64_t id = xcd_tile(workgroup(), mtiles * ntiles);
        if (id < 0) return;
        constexpr int GM = 8;
        const int64_t strip = id / (GM * ntiles), in = id % (GM * ntiles);
        const int64_t gm = mtiles - strip * GM < GM ? mtiles - strip * GM : GM;
        nt = in / gm;
        r0 = (strip * GM + in % gm) * BM;
        nrows = a.rows - r0 < BM ? a.rows - r0 : BM;
    } else {
        // only the workgroups that have a tile come past this (no barrier yet)
        const bool rest = !SPLITS || a.splits == 1;
        TileAt none;
        const int64_t tiles = scalar(find_tile(a.offsets, a.G, a.M, BM, a.skip, rest, -1, none));
        const int64_t id = xcd_tile(workgroup(), tiles * ntiles);
        if (id < 0) return;
        nt = id % ntiles;
        find_tile(a.offsets, a.G, a.M, BM, a.skip, rest, id / ntiles, t);
        t.g = __builtin_amdgcn_readfirstlane(t.g);
        t.p0 = scalar(t.p0);
        t.p1 = scalar(t.p1);
        r0 = t.p0;
        nrows = t.p1 - t.p0;
    }
    const int64_t c0 = nt * BN;
    const bool rest = KIND != kDw && a.offsets != nullptr && t.g == a.G;

    // the part of the sum that this split takes, in tiles
    const int64_t kall = ka > kb ? ka : kb;
    int64_t steps = (kall + BK - 1) / BK;
    if (SPLITS && a.splits > 1) {
        const int64_t each = (steps + a.splits - 1) / a.splits;
        kbeg = split * each * BK;
        const int64_t left = steps - split * each;
        steps = left < each ? (left > 0 ? left : 0) : each;
    }
    if (rest) steps = 0;
    // what is left of the sum from tile i on, in A and in B
    const int64_t kend = kbeg + steps * BK;
    const int64_t ea = ka < kend ? ka : kend, eb = kb < kend ? kb : kend;
    auto left = [&](int64_t end, int64_t i) {
        const int64_t r = end - kbeg - i * BK;
        return r > BK ? BK : (int)r;
    };

    OpA oa;
    OpB ob;
    const T *Bg = (const T *)a.B + (KIND == kDw || rest ? 0 : (int64_t)t.g * a.gsb);
    if constexpr (AKM) oa.init_km((const T *)a.A, a.lda, a.amap, r0, nrows, kbeg);
    else oa.init_mn((const T *)a.A, a.lda, a.amap, r0, a.rows, pos, kbeg);
    if constexpr (BKM) {
        const RowMap id{nullptr, 0, 0, 0};
        ob.init_km(Bg, a.ldb, id, c0, a.N - c0 < BN ? a.N - c0 : BN, kbeg);
    } else {
        ob.init_mn(Bg, a.ldb, a.bmap, c0, a.N, pos, kbeg);
    }

    // acc[i][j]: row block i of A's first part (i < TB) or second, column block
    // j likewise
    v16f acc[2 * TB][2 * TB];
#pragma unroll
    for (int i = 0; i < 2 * TB; ++i)
#pragma unroll
        for (int j = 0; j < 2 * TB; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const int wm = (wave >> 1) * (TB * 32), wn = (wave & 1) * (TB * 32);
    // A's first and second part; of B's, tiles take turns in which holds the first
    typename Mma<T>::Frag fa[2][4][TB], fb[2][4][TB];
    auto read_a = [&](int to, Lds part, int n) { fa[to][n / TB][n % TB] = OpA::frag(part, wm + n % TB * 32, n / TB); };
    auto read_b = [&](int to, Lds part, int n) { fb[to][n / TB][n % TB] = OpB::frag(part, wn + n % TB * 32, n / TB); };
    // All but the latest `later` loads to LDS have arrived, in every wave
    // (vmcnt, which counts a wave's loads in order; the other counters are left
    // alone), and every wave has read what it read (the compiler's wait before
    // the barrier).  The compiler does not know what the loads in assembly write,
    // so what keeps them apart from the reads of the same place is that one of
    // these barriers, which no access to LDS crosses, lies between them both ways.
    // Nothing but loads to LDS is under way in the loop: another load among them
    // can only make the wait longer.
    auto landed = [&](auto later) {
        constexpr int n = decltype(later)::value;
        __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
        __syncthreads();
    };
    // A quarter: A's part I with what fb[B] holds, as B's part J; between the
    // products the reads of a part and `loads` loads, in this order.
    auto quarter = [&](auto I, auto B, auto J, auto read, auto load) {
        constexpr int i0 = decltype(I)::value, b = decltype(B)::value, j0 = decltype(J)::value;
        constexpr int PRODUCTS = 4 * TB * TB, READS = 4 * TB;
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) {
            const int s = n / (TB * TB), i = n / TB % TB, j = n % TB;
            acc[i0 * TB + i][j0 * TB + j] = Mma<T>::m32(fb[b][s][j], fa[i0][s][i], acc[i0 * TB + i][j0 * TB + j]);
            // the reads in the first half, so that a barrier at the quarter's end
            // finds them done
#pragma unroll
            for (int r = 2 * n * READS / PRODUCTS; r < 2 * (n + 1) * READS / PRODUCTS && r < READS; ++r) read(r);
#pragma unroll
            for (int l = n * IT / PRODUCTS; l < (n + 1) * IT / PRODUCTS; ++l) load(l);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    std::integral_constant<int, 0> c0_;
    std::integral_constant<int, 1> c1_;
    auto place_a = [&](int odd, int part) { return parts + (odd * 2 + part) * PART; };
    auto place_b = [&](int odd, int part) { return parts + (4 + odd * 2 + part) * PART; };
    auto send_rows = [&](int64_t i) {
        if constexpr (KIND == kDw) {
            oa.send_rows(i, kbeg + i * BK, ka);
            ob.send_rows(i, kbeg + i * BK, kb);
        }
    };
    auto read_rows = [&](int64_t i) {
        if constexpr (KIND == kDw) {
            oa.read_rows(i);
            ob.read_rows(i);
        }
    };
    auto take_rows = [&]() {
        if constexpr (KIND == kDw) {
            oa.take_rows();
            ob.take_rows();
        }
    };
    // Tile i (odd: ODD): on entry fa[0] and fb[ODD] hold A0 and B0, on exit
    // those of the next tile (the latter in fb[!ODD]).  END: the tiles it
    // sends for may lie past the end of the sum.
    auto tile = [&](auto ODD, auto END, int64_t i) {
        constexpr int odd = decltype(ODD)::value;
        constexpr bool end = decltype(END)::value;
        std::integral_constant<int, 1 - odd> other;
        take_rows();
        send_rows(i + 4);
        const char *from_a = (const char *)scalar((int64_t)(oa.base + (i + 2) * oa.adv));
        const char *from_b = (const char *)scalar((int64_t)(ob.base + (i + 2) * ob.adv));
        const int ra = end ? left(ea, i + 2) : 0, rb = end ? left(eb, i + 2) : 0;
        auto load_a = [&](int half, int l) {
            if (end) oa.issue_end(from_a, place_a(odd, half), wave, half, l, ra);
            else oa.issue(from_a, place_a(odd, half), wave, half, l);
        };
        auto load_b = [&](int half, int l) {
            if (end) ob.issue_end(from_b, place_b(odd, half), wave, half, l, rb);
            else ob.issue(from_b, place_b(odd, half), wave, half, l);
        };
        quarter(c0_, ODD, c0_, [&](int n) { read_b(1 - odd, place_b(odd, 1), n); }, [&](int l) { load_a(0, l); });
        quarter(c0_, other, c1_, [&](int n) { read_a(1, place_a(odd, 1), n); }, [&](int l) { load_b(0, l); });
        landed(std::integral_constant<int, 4 * IT>{});
        read_rows(i + 3);
        quarter(c1_, other, c1_, [&](int n) { read_a(0, place_a(1 - odd, 0), n); }, [&](int l) { load_b(1, l); });
        quarter(c1_, ODD, c0_, [&](int n) { read_b(1 - odd, place_b(1 - odd, 0), n); }, [&](int l) { load_a(1, l); });
        landed(std::integral_constant<int, 4 * IT>{});
    };
    if (steps > 0) {
        if constexpr (KIND == kDw) {
            oa.ring = (typename OpA::Ring)rings + wave * 2 * OpA::kRing;
            ob.ring = (typename OpB::Ring)rings + (wave * 2 + 1) * OpB::kRing;
            if (oa.map.slots != nullptr || ob.map.slots != nullptr) {
                for (int i = 0; i < 4; ++i) send_rows(i);
                landed(c0_);
            }
        }
        // both tiles' parts in the order of their use
        for (int i = 0; i < 2; ++i) {
            read_rows(i);
            take_rows();
            const char *from_a = oa.base + i * oa.adv, *from_b = ob.base + i * ob.adv;
            const int ra = left(ea, i), rb = left(eb, i);
#pragma unroll
            for (int l = 0; l < IT; ++l) oa.issue_end(from_a, place_a(i, 0), wave, 0, l, ra);
#pragma unroll
            for (int l = 0; l < IT; ++l) ob.issue_end(from_b, place_b(i, 0), wave, 0, l, rb);
#pragma unroll
            for (int l = 0; l < IT; ++l) ob.issue_end(from_b, place_b(i, 1), wave, 1, l, rb);
#pragma unroll
            for (int l = 0; l < IT; ++l) oa.issue_end(from_a, place_a(i, 1), wave, 1, l, ra);
        }
        read_rows(2);
        landed(std::integral_constant<int, 6 * IT>{});
#pragma unroll
        for (int n = 0; n < 4 * TB; ++n) {
            read_a(0, place_a(0, 0), n);
            read_b(0, place_b(0, 0), n);
        }
        landed(std::integral_constant<int, 4 * IT>{});
        // two tiles a round; of an odd number the last one's partner is zeros,
        // multiplied all the same with tiles of 256, whose registers the branch
        // would spill
        const int64_t whole = (ea < eb ? ea : eb) - kbeg;  // steps of the sum in both
        int64_t i = 0;
        for (; (i + 4) * BK <= whole; i += 2) {
            tile(c0_, std::false_type{}, i);
            tile(c1_, std::false_type{}, i + 1);
        }
        for (; i < steps; i += 2) {
            tile(c0_, std::true_type{}, i);
            if (BS == 256 || i + 1 < steps) tile(c1_, std::true_type{}, i + 1);
        }
    }
    const int lane = threadIdx.x & 63;
    constexpr bool PLAIN = KIND != kFwd && sizeof(T) == 2;
    if constexpr (PLAIN) {
        // ---- out, without an epilogue: the wave's block, rounded, goes through
        // LDS at once, so that the rows leave in whole chunks.  A lane holds one
        // row of C and 4 columns apiece of it (the operands are multiplied the
        // other way round).  Chunk c of row r lies at place c ^ r, so that
        // neither the lanes that write one chunk of many rows nor those that
        // read a row meet on a bank.
        if (!SPLITS || a.splits == 1) {
            constexpr int CH = TB * 8;       // 16-byte chunks of a row
            constexpr int ROWS = TB * 64;
            constexpr int RPP = 64 / CH;     // rows that a wave writes at once
            static_assert(4 * ROWS * CH * 16 <= sizeof(smem), "the staged rows fit the tiles");
            typedef T Four __attribute__((ext_vector_type(4)));
            T *stage = smem + wave * ROWS * CH * E;
            landed(c0_);
#pragma unroll
            for (int i = 0; i < 2 * TB; ++i)
#pragma unroll
                for (int j = 0; j < 2 * TB; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        Four v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = (T)acc[i][j][q * 4 + e];
                        const int row = i * 32 + (lane & 31);
                        *(Four *)(stage + (row * CH + ((j * 4 + q) ^ (row & (CH - 1)))) * E + (lane >> 5) * 4) = v;
                        // (a few accumulators at a time: all at once do not fit)
                        __builtin_amdgcn_sched_barrier(0);
                    }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const int lc = lane % CH;
            const int64_t col = c0 + lc / (CH / 2) * (BN / 2) + wn + lc % (CH / 2) * 8;
            const int64_t gone = a.N - col;
            const int n = gone >= 8 ? 8 : (gone > 0 ? (int)gone : 0);
            T *out = (T *)a.C + (rest ? 0 : (int64_t)t.g * a.gsc) + col;
            const bool sure = nrows == BM && c0 + BN <= a.N && a.chunked;
#pragma unroll 1
            for (int q = 0; q < ROWS; q += 8 * RPP) {
                Chunk<T, E> v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = q + k * RPP + lane / CH;
                    v[k].load(stage + (row * CH + (lc ^ (row & (CH - 1)))) * E);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = q + k * RPP + lane / CH;
                    const int64_t r = row / (TB * 32) * (BM / 2) + wm + row % (TB * 32);
                    if (!sure && (r >= nrows || n == 0)) continue;
                    T *to = out + (KIND == kDw ? r0 + r : a.cmap(r0 + r)) * a.ldc;
                    if (sure || (n == 8 && a.chunked)) {
                        v[k].store(to);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < n) to[e] = v[k].e[e];
                    }
                }
            }
            return;
        }
    }
    if constexpr (!PLAIN || SPLITS) {
    // ---- out: one part's rows of a wave at a time through LDS, so that the
    // rows leave in whole chunks.  A lane holds one row of C and 4 columns
    // apiece of it (the operands are multiplied the other way round).  Chunk c
    // of row r lies at place c ^ r: both the lanes that write one chunk of many
    // rows and those that read a row meet different banks.
    constexpr int CH = TB * 16;          // 16-byte chunks of a staged row
    constexpr int LPR = CH / 2;          // lanes that write a row of C
    constexpr int RPP = 64 / LPR;        // rows that a wave writes at once
    constexpr int ROWS = TB * 32;        // rows of a part
    // rows a lane takes at a time (with four, tiles of 128 spill)
    constexpr int BATCH = BS == 128 ? 2 : 4;
    static_assert(4 * ROWS * CH * 16 <= sizeof(smem), "the staged rows fit the tiles");
    v4f *stage = reinterpret_cast<v4f *>(smem) + wave * ROWS * CH;
    Epilogue<T> ep;
    // the first half of a row's lanes: the wave's columns in B's first part
    const int lc = lane % LPR;
    const int64_t col = c0 + lc / (LPR / 2) * (BN / 2) + wn + lc % (LPR / 2) * 8;
    if (KIND != kFwd || (SPLITS && a.splits > 1) || rest) {
        ep.col = col;
        const int64_t left = a.N - col;
        ep.n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    } else {
        ep.init(a, t.g, col);
    }
    auto put_part = [&](auto P) {
        constexpr int p = decltype(P)::value;
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
            for (int j = 0; j < 2 * TB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v4f v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[p * TB + i][j][q * 4 + e];
                    const int row = i * 32 + (lane & 31), c = j * 8 + q * 2 + (lane >> 5);
                    stage[row * CH + (c ^ (row & (CH - 1)))] = v;
                    __builtin_amdgcn_sched_barrier(0);
                }
    };
    // every row and column of the tile exists, on whole chunks
    const bool sure = nrows == BM && c0 + BN <= a.N && a.chunked && !rest && (!SPLITS || a.splits == 1);
    auto row_at = [&](int p, int q, int k) {
        const int64_t r = r0 + p * (BM / 2) + wm + lane / LPR + q + k * RPP;
        return KIND == kDw ? r : a.cmap(r);
    };
    // the residual of a batch, sent for a batch ahead
    typename Epilogue<T>::Eight res[BATCH];
    const bool added = KIND == kFwd && sure && a.R != nullptr;
    auto send_for = [&](int p, int q) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            res[k].load((const T *)a.R + row_at(p, q, k) * a.ldr + col);
        }
    };
    // the tiles are read to the end, and no load to LDS is under way; only then
    // the first batch's residual is sent for, whose loads are the compiler's and
    // so not to be counted on in a wait (they are back by the time the first
    // part is staged)
    landed(c0_);
    if (added) send_for(0, 0);
#pragma unroll 1
    for (int p = 0; p < 2; ++p) {
        // (the empty statements keep the compiler from making one block of the
        // two, which would select between all the accumulators)
        if (p == 0) {
            asm volatile("; first part");
            put_part(c0_);
            asm volatile("; first part staged");
        } else {
            asm volatile("; second part");
            put_part(c1_);
            asm volatile("; second part staged");
        }
        // the wave's own region: its lanes' writes before its lanes' reads
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int64_t p0 = p * (BM / 2) + wm + lane / LPR;
#pragma unroll 1
        for (int q = 0; q < ROWS; q += BATCH * RPP) {
            float v[BATCH * 8];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int row = q + k * RPP + lane / LPR;
                const v4f lo = stage[row * CH + ((lc * 2) ^ (row & (CH - 1)))];
                const v4f hi = stage[row * CH + ((lc * 2 + 1) ^ (row & (CH - 1)))];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[k * 8 + e] = lo[e];
                    v[k * 8 + 4 + e] = hi[e];
                }
            }
            if (SPLITS && a.splits > 1) {
                const int64_t all = KIND == kDw ? (int64_t)a.G * a.rows : a.M;
                const int64_t first = split * all + (KIND == kDw ? (int64_t)t.g * a.rows : 0) + r0;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int64_t r = p0 + q + k * RPP;
                    if (r < nrows)
                        Epilogue<float>::put(a.part + (first + r) * a.N + col, *(const float(*)[8])(v + k * 8), ep.n);
                }
                continue;
            }
            int64_t crow[BATCH];
            if (sure) {
                typename Epilogue<T>::Eight now[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    crow[k] = row_at(p, q, k);
                    now[k] = res[k];
                }
                if (added) {
                    if (q + BATCH * RPP < ROWS) send_for(p, q + BATCH * RPP);
                    else if (p == 0) send_for(1, 0);
                }
                ep.template out<true, KIND != kFwd>(a, t.g, crow, v, now);
                continue;
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) crow[k] = p0 + q + k * RPP < nrows ? row_at(p, q, k) : -1;
            if (rest) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k)
                    if (crow[k] >= 0) ep.zero(a, crow[k]);
            } else {
                ep.template out<false, KIND != kFwd>(a, t.g, crow, v, nullptr);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    }
}

// Adds the partial products of a split sum and runs the epilogue: 8 columns a
// thread, the splits in order.
template <typename T>
__global__ __launch_bounds__(256) void k_join(LinArgs a, int kind) {
    const int64_t all = kind == kDw ? (int64_t)a.G * a.rows : a.M;
    const int64_t chunks = (a.N + 7) / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= all * chunks) return;
    const int64_t r = id / chunks, col = id % chunks * 8;
    int g = 0;
    int64_t crow = r;
    bool rest = false;
    if (kind == kDw) {
        g = (int)(r / a.rows);
        crow = r % a.rows;
    } else {
        crow = a.cmap(r);
        if (a.offsets != nullptr) {
            // the last group that starts at or before r and is not empty
            int lo = 0, hi = a.G;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (group_at(a.offsets, mid + 1, a.M) <= r) lo = mid + 1;
                else hi = mid;
            }
            g = lo;
            rest = g >= a.G;
            if (!rest) {
                const int64_t n = group_at(a.offsets, g + 1, a.M) - group_at(a.offsets, g, a.M);
                if (n <= a.skip) return;
            }
        }
    }
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    Epilogue<T> ep;
    if (rest) {
        ep.n = a.N - col >= 8 ? 8 : (int)(a.N - col);
        ep.col = col;
        ep.zero(a, crow);
        return;
    }
    ep.init(a, g, col);
    for (int s = 0; s < a.splits; ++s) {
        float w[8];
        Epilogue<float>::get(a.part + ((int64_t)s * all + r) * a.N + col, w, ep.n);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += w[i];
    }
    const int64_t rows[1] = {crow};
    ep.template out<false, false>(a, g, rows, v, nullptr);
}

// ---- a few rows against a whole weight matrix -----------------------------------------
//
// Up to 16 rows, those that one matrix instruction takes.  Bound by the stream
// of the weights.  A workgroup takes NT blocks of 16 rows of W (columns of C);
// its waves take every WV-th run of U steps of the sum and read W straight into
// the matrix instruction's registers, 16 bytes a lane, all loads of a run in
// flight; the rows of X come from cache, and rows that do not exist are not
// read.  The waves' sums are added in wave order through LDS.  Groups of more
// rows are left to the tiled product.
//
// bf16, weights from memory: one row by 16384 x 4096 26 us (5.2 TB/s; the
// tiled product 40), 16 rows 34 us (40); 16 rows by 4096 x 4096 13 us (18).
// More blocks of rows or 8 waves gained nothing.  Rows that are no whole 16-byte
// chunks are read element by element, each load waited for: one row by 16384 x
// 4095 125 us.
template <typename T, int NT, int WV, bool WIDE>
__global__ __launch_bounds__(WV * 64) void k_product_few(LinArgs a) {
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int STEP = 4 * E;  // elements of the sum in one load of a wave
    __shared__ float sm[WV][16][NT * 16 + 1];
    const int g = blockIdx.y;
    int64_t p0 = 0, cnt = a.M;
    if (a.offsets != nullptr) {
        p0 = group_at(a.offsets, g, a.M);
        cnt = group_at(a.offsets, g + 1, a.M) - p0;
        if (cnt <= 0 || cnt > a.skip) return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (NT * 16);
    const T *w[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t n = n0 + t * 16 + l;
        w[t] = (const T *)a.B + (int64_t)g * a.gsb + (n < a.N ? n : a.N - 1) * a.ldb;
    }
    const bool xin = l < cnt;
    const T *x = (const T *)a.A + a.amap(p0 + (xin ? l : 0)) * a.lda;
    v4f acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    typedef typename Mma<T>::Frag Frag;
    const int K = (int)a.ka;
    auto load = [&](const T *p, int k, bool in) {
        Frag f;
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = (T)0.0f;
        if constexpr (WIDE) {
            if (in && k < K) f = *reinterpret_cast<const Frag *>(p + k);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (in && k + i < K) f[i] = p[k + i];
        }
        return f;
    };
    constexpr int U = 4;  // steps of the sum a wave has in flight
    for (int k0 = wave * STEP * U; k0 < K; k0 += WV * STEP * U) {
        Frag fw[U][NT], fx[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) fw[u][j] = load(w[j], k0 + u * STEP + q * E, true);
#pragma unroll
        for (int u = 0; u < U; ++u) fx[u] = load(x, k0 + u * STEP + q * E, xin);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] = Mma<T>::m16(fw[u][j], fx[u], acc[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sm[wave][l][j * 16 + q * 4 + i] = acc[j][i];
    __syncthreads();
    // 8 columns a thread
    for (int i = threadIdx.x; i < 16 * NT * 2; i += WV * 64) {
        const int m = i / (NT * 2), c = i % (NT * 2) * 8;
        if (m >= cnt) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = 0.0f;
            for (int k = 0; k < WV; ++k) v[e] += sm[k][m][c + e];
        }
        Epilogue<T> ep;
        ep.init(a, g, n0 + c);
        const int64_t rows[1] = {a.cmap(p0 + m)};
        ep.template out<false, false>(a, g, rows, v, nullptr);
    }
}

// ---- the backward pass's element-wise step ----------------------------------------------
//
// dZ[p] = dY[slot(p)] act'(z[slot(p)]) in position order, rounded to the type
// that the matrix instructions take (and padded with zeros to whole chunks),
// and the partial column sums of the unrounded values for db: one row tile of
// one group (there are `most` of them at most) and 8 columns a thread.
//
// Bound by memory.  Workgroups in turn take neighbouring columns of the same
// rows, so that whole rows are read together: with neighbouring rows' pieces of
// 512 bytes instead, 32768 x 4096 in bf16 with a thin dX took 291 against 261
// us by slots and 248 against 229 without (16384 x 4096, half of which the last
// cache holds, 133 against 137).
constexpr int kGradRows = 64;
template <typename T>
__global__ __launch_bounds__(256) void k_act_grad(LinArgs a, const void *dY, int64_t ldd, int df32, T *dZ, int64_t lddz,
                                                  float *colsum, int64_t most) {
    __shared__ float sm[8][256];
    const unsigned cols = (unsigned)((a.N + 255) / 256);
    const int64_t id = workgroup();
    const int64_t tile = id / cols, stripe = id % cols;
    if (tile >= most) return;
    TileAt t{0, 0, 0};
    if (a.offsets == nullptr) {
        t.p0 = tile * kGradRows;
        t.p1 = t.p0 + kGradRows < a.M ? t.p0 + kGradRows : a.M;
    } else {
        find_tile(a.offsets, a.G, a.M, kGradRows, 0, false, tile, t);
        if (t.g < 0) return;
    }
    // 32 threads across 256 columns, 8 rows at a time
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int64_t col = stripe * 256 + cx * 8;
    const int n = a.N - col >= 8 ? 8 : (a.N > col ? (int)(a.N - col) : 0);
    const int npad = lddz - col >= 8 ? 8 : (lddz > col ? (int)(lddz - col) : 0);
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    // SURE: all rows and columns of the tile exist, on whole chunks.  One row of
    // the thread's eight at a time: several together cost waves, and with them
    // time (32768 x 4096: one 251 us with a thin dX, four 265).
    auto rows = [&](auto sure) {
        constexpr bool SURE = decltype(sure)::value;
#pragma unroll 1
        for (int64_t p = t.p0 + ry; p < t.p1; p += 8) {
            const int64_t row = a.cmap(p);
            float d[8], z[8];
            if (df32) Epilogue<float>::template get<SURE>((const float *)dY + row * ldd + col, d, n);
            else Epilogue<T>::template get<SURE>((const T *)dY + row * ldd + col, d, n);
            if (a.act != FK_ACT_NONE) {
                Epilogue<T>::template get<SURE>((const T *)a.Z + row * a.ldz + col, z, n);
                times_slope<sizeof(T) == 4>(a.act, z, d);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = SURE || i < n ? d[i] : 0.0f;
                s[i] += d[i];
            }
            if (dZ != nullptr) Epilogue<T>::template put<SURE>(dZ + p * lddz + col, d, npad);
        }
    };
    if (a.chunked && t.p1 - t.p0 == kGradRows && (stripe + 1) * 256 <= a.N) rows(std::true_type{});
    else if (n > 0 || (dZ != nullptr && npad > 0)) rows(std::false_type{});
    if (colsum == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sm[ry][cx * 8 + i] = s[i];
    __syncthreads();
    const int64_t c = stripe * 256 + threadIdx.x;
    if (c < a.N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += sm[i][threadIdx.x];
        colsum[tile * a.N + c] = v;
    }
}

// db of one group: its row tiles' column sums in order, 16 threads down a
// column.  There are `most` row tiles at most; offsets that do not rise cannot
// reach past them.
template <typename T>
__global__ __launch_bounds__(256) void k_bias_grad(LinArgs a, const float *colsum, int64_t most, void *db, int f32) {
    __shared__ float sm[16][17];
    __shared__ int64_t range[2];
    const int g = blockIdx.y;
    if (threadIdx.x < 64) {
        int64_t first = 0, tiles;
        if (a.offsets == nullptr) {
            tiles = (a.M + kGradRows - 1) / kGradRows;
        } else {
            // the row tiles of the groups before this one
            int64_t s = 0;
            for (int i = threadIdx.x; i < g; i += 64) {
                const int64_t c = group_at(a.offsets, i + 1, a.M) - group_at(a.offsets, i, a.M);
                s += c > 0 ? (c + kGradRows - 1) / kGradRows : 0;
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) s += __shfl_xor(s, o, 64);
            first = s;
            const int64_t c = group_at(a.offsets, g + 1, a.M) - group_at(a.offsets, g, a.M);
            tiles = c > 0 ? (c + kGradRows - 1) / kGradRows : 0;
        }
        if (threadIdx.x == 0) {
            range[0] = first;
            range[1] = first + tiles < most ? first + tiles : most;
        }
    }
    __syncthreads();
    const int col = threadIdx.x & 15, down = threadIdx.x >> 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    float s = 0.0f;
    if (c < a.N) {
#pragma unroll 4
        for (int64_t p = range[0] + down; p < range[1]; p += 16) s += colsum[p * a.N + c];
    }
    sm[down][col] = s;
    __syncthreads();
    if (down == 0 && c < a.N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += sm[i][col];
        const int64_t at = (int64_t)g * a.N + c;
        if (f32) ((float *)db)[at] = v;
        else ((T *)db)[at] = (T)v;
    }
}

// out[r] = in[map(r)] with its columns padded by zeros to ldo (whole chunks): the
// tiled product reads 16 bytes at a time, so operands whose rows do not start
// on 16 bytes are laid out once more first, both of a product in one launch.
// 2^lx lanes across a row's chunks.
struct PadJob {
    const void *in;
    void *out;
    RowMap map;
    int64_t rows, ldi, ldo;
    int cols, lx;
};
template <typename T>
__global__ __launch_bounds__(256) void k_pad_rows(PadJob j0, PadJob j1) {
    constexpr int E = 16 / (int)sizeof(T);
    const PadJob j = blockIdx.y ? j1 : j0;
    const int tx = threadIdx.x & ((1 << j.lx) - 1), ty = threadIdx.x >> j.lx;
    const int rpb = 256 >> j.lx;
    for (int64_t r = (int64_t)blockIdx.x * rpb + ty; r < j.rows; r += (int64_t)gridDim.x * rpb) {
        const T *p = (const T *)j.in + j.map(r) * j.ldi;
        T *q = (T *)j.out + r * j.ldo;
        for (int64_t c = (int64_t)tx * E; c < j.ldo; c += (int64_t)E << j.lx) {
            Chunk<T, E> o;
#pragma unroll
            for (int i = 0; i < E; ++i) o.e[i] = c + i < j.cols ? p[c + i] : (T)0.0f;
            o.store(q + c);
        }
    }
}

// ---- host ---------------------------------------------------------------------------------

constexpr int kFewRows = 16;  // most rows of a group that k_product_few takes
constexpr int kCus = 256;

// Whether eight columns from a multiple of eight on are whole 16-byte chunks.
bool on_chunks(const void *p, int64_t ld, size_t size) {
    return p == nullptr || (((uintptr_t)p & 15) == 0 && ld * (int64_t)size % 16 == 0);
}

template <typename T, int KIND>
hipError_t run_product(LinArgs a, int tile, hipStream_t s) {
    a.chunked = on_chunks(a.C, a.ldc, a.cf32 ? 4 : sizeof(T)) && on_chunks(a.C, a.gsc, a.cf32 ? 4 : sizeof(T)) &&
                on_chunks(a.R, a.ldr, sizeof(T)) && on_chunks(a.Z, a.ldz, sizeof(T));
    const int64_t nt = cdiv(a.N, tile);
    int64_t mt, grid;
    if (KIND == kDw) {
        mt = cdiv(a.rows, tile);
        grid = (mt * nt + 7) / 8 * 8 * a.G;
    } else if (a.offsets == nullptr) {
        mt = cdiv(a.rows, tile);
        grid = mt * nt;
    } else {
        // the groups that have tiles hold more than skip rows each
        const int64_t most = a.M / (a.skip + 1);
        mt = a.M / tile + (most < a.G ? most : a.G) + 1;
        grid = mt * nt;
    }
    if (grid > 0) {
        if (grid > INT32_MAX) return hipErrorInvalidValue;
        const dim3 gr = long_grid(grid, a.splits);
        if constexpr (sizeof(T) == 2) {
            if (tile == 256) k_product<T, KIND, 256><<<gr, kTileThreads, 0, s>>>(a, mt, nt);
        }
        if (tile == 128) k_product<T, KIND, 128><<<gr, kTileThreads, 0, s>>>(a, mt, nt);
    }
    if (a.splits > 1) {
        const int64_t all = KIND == kDw ? (int64_t)a.G * a.rows : a.M;
        const int64_t n = cdiv(all * cdiv(a.N, 8), 256);
        if (n > INT32_MAX) return hipErrorInvalidValue;
        if (n > 0) k_join<T><<<(unsigned)n, 256, 0, s>>>(a, KIND);
    }
    return hipGetLastError();
}

template <typename T, bool WIDE>
hipError_t run_few(const LinArgs &a, hipStream_t s) {
    // 32 columns a workgroup where there are many of them.  bf16: 64 groups of
    // 1 to 16 rows of 4096 x 2048, 8 on average: 205 us against 231 with 16
    // columns; one row by 16384 x 4096 (1024 workgroups of 16): 38 against 28.
    const int groups = a.offsets ? a.G : 1;
    if (cdiv(a.N, 16) * groups >= 4096) {
        k_product_few<T, 2, 4, WIDE><<<dim3((unsigned)cdiv(a.N, 32), (unsigned)groups), 256, 0, s>>>(a);
    } else {
        k_product_few<T, 1, 4, WIDE><<<dim3((unsigned)cdiv(a.N, 16), (unsigned)groups), 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

// Tile and splits of a product of `groups` matrices of rows x cols with sums
// of `steps` 128-byte steps.
//
// Tiles of 256 read half as much a product as those of 128 and run at 1350
// TFLOP/s where those reach 1100 (bf16, 16384 x 8192 x 4096), if there are
// enough of them: on 256 CUs, 160 tiles of 256 took 80 us forward and 170 for
// both gradients (4096 x 2560 x 4096) against 86 and 206 for four times as many
// of 128; 128 tiles of 256 took 76, 67 and 86 (forward, dX, dW) against 63, 75
// and 84.  (Of short sums with gelu and a residual, tiles of 128 are ahead at
// more tiles too, two workgroups of a CU covering each other's epilogues: 160 of
// 256 by a sum of 512 38 us against 31, 256 of them 44 against 40.)  In fp32,
// whose matrix instructions take 16 times as long, tiles of 128 are never
// starved: 8192 x 8192 x 2048 1908, 1899 and 1909 us against 1950, 1926 and
// 2142, 4096 x 5120 x 1024 365, 298 and 471 against 503, 1197 and 1050.
//
// A sum is split where the tiles leave CUs without work.  In units of a step's
// time in bf16 (about 0.4 us with a workgroup a CU): the join's launch costs 8,
// its partial tiles, written and read, 1/8 each; fp32's steps take four times
// as long and more, and those of a single row tile, whose other operand comes
// from memory, twice (32 rows by 16384 x 4096, 128 tiles of 64 steps: 45 us,
// in two splits 41).  In fp32, where a CU's workgroups take turns at its matrix
// units, an uneven last round is evened out too.  Measured in bf16 with 1, 2, 4
// and 8 splits (us): 32 tiles of 64 steps 27, 21, 19, 22; 64 tiles of 64 steps
// 28, 24, 28, 32; 128 tiles of 64 steps 30, 34 (two), 64 tiles of 256 steps 92,
// 61, 55, 64; 64 tiles of 32 steps 16, 19, 22, 28.
struct Shape {
    int tile, splits;
};
Shape pick_shape(int64_t rows, int64_t cols, int64_t groups, int64_t steps, int dtype) {
    const bool f32 = dtype == FK_F32;
    Shape s;
    const int64_t big = cdiv(rows, 256) * cdiv(cols, 256) * groups;
    s.tile = !f32 && rows > 128 && big >= kCus * 5 / 8 ? 256 : 128;
    s.splits = 1;
    if (s.tile == 256) return s;
    const int64_t tiles = cdiv(rows, 128) * cdiv(cols, 128) * groups;
    const int64_t unit = 8 * (f32 ? 4 : rows <= 128 ? 2 : 1);  // (costs in eighths)
    const int64_t most = f32 ? 4 * kCus : kCus;
    int64_t best = cdiv(tiles, kCus) * steps * unit;
    for (int n = 2; n <= 32 && n <= steps && tiles * n <= most; ++n) {
        const int64_t cost = cdiv(tiles * n, kCus) * cdiv(steps, n) * unit + 64 + tiles * n;
        if (cost < best) best = cost, s.splits = n;
    }
    return s;
}

size_t pad16(int64_t rows, int64_t cols, int dtype) {
    const int64_t e = 16 / (int64_t)dtype_size(dtype);
    return align_up((size_t)rows * (size_t)(cdiv(cols, e) * e) * dtype_size(dtype), 256);
}

bool whole(int64_t cols, int64_t ld, int dtype) {
    const int64_t e = 16 / (int64_t)dtype_size(dtype);
    return cols % e == 0 && ld % e == 0;
}

// The tiled product reads an operand as it lies if its rows are whole chunks
// and the 32-bit offsets of its loads reach: over a tile's rows from the
// tile's first, or, where slots say which rows, over the whole matrix (with
// 2 GB to spare for what is added within a row).
constexpr int64_t kReach = (int64_t)1 << 31;
bool readable(int64_t cols, int64_t ld, int dtype) {
    return whole(cols, ld, dtype) && ld * 256 * (int64_t)dtype_size(dtype) <= kReach;
}
bool reachable(int64_t rows, int64_t ld, int dtype) {
    return (double)rows * (double)ld * (double)dtype_size(dtype) <= (double)kReach;
}

}  // namespace

// What a call needs and in which order its scratch is laid out.
LinearPlan plan_linear(const LinearShape &h, bool backward) {
    LinearPlan p{};
    p.M = h.M, p.G = h.grouped ? h.G : 0;
    const int64_t groups = h.grouped ? h.G : 1;
    const int64_t bk = 128 / (int64_t)dtype_size(h.dtype);
    const int64_t mean = h.grouped ? cdiv(h.M, h.G) : h.M;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += align_up(bytes > 0 ? bytes : 1, 256);
        return o;
    };
    // in groups only where few are likely to be left to the tiled product, which
    // then runs too: 64 groups of 4096 x 2048 with 8 rows on average 205 us (the
    // tiled product alone 214), with 16 on average 235 (217)
    p.few = !backward && mean <= (h.grouped ? kFewRows / 2 : kFewRows);
    p.tiled = backward || h.grouped || !p.few;
    const int64_t kp = cdiv(h.K, bk / 8) * (bk / 8);
    p.pad_x = p.tiled && !readable(h.K, h.ldx, h.dtype);
    p.pad_w = p.tiled && !readable(h.K, h.ldw, h.dtype);
    // X by slots past the loads' reach: laid out in position order
    p.sort_x = p.tiled && h.by_slots && !reachable(h.M / h.share, p.pad_x ? kp : h.ldx, h.dtype);
    p.pad_x = p.pad_x || p.sort_x;
    const int64_t wrows = groups * h.N;
    if (p.pad_x) p.xpad = take(pad16(p.sort_x ? h.M : h.M / h.share, h.K, h.dtype));
    if (p.pad_w) p.wpad = take(pad16(wrows, h.K, h.dtype));
    if (!backward) {
        const Shape s = pick_shape(h.grouped ? mean : h.M, h.N, groups, cdiv(h.K, bk), h.dtype);
        p.tile = s.tile, p.splits = s.splits;
        if (p.tiled && p.splits > 1) p.part = take((size_t)p.splits * h.M * h.N * 4);
        p.total = off > 0 ? off : 256;
        return p;
    }
    // dZ is laid out in position order unless dY serves as it is
    p.make_dz = h.act != FK_ACT_NONE || h.ydtype != h.dtype || !readable(h.N, h.ldy, h.dtype) ||
                (h.by_slots && !reachable(h.M, h.ldy, h.dtype));
    if (p.make_dz) p.dz = take(pad16(h.M, h.N, h.dtype));
    p.grad_tiles = h.grouped ? h.M / kGradRows + (h.G < h.M ? h.G : h.M) : cdiv(h.M, kGradRows);
    p.colsum = take((size_t)p.grad_tiles * h.N * 4);
    const Shape sx = pick_shape(h.grouped ? mean : h.M, h.K, groups, cdiv(h.N, bk), h.dtype);
    const Shape sw = pick_shape(h.N, h.K, groups, cdiv(mean, bk), h.dtype);
    p.tile = sx.tile, p.splits = sx.splits, p.tile_w = sw.tile, p.splits_w = sw.splits;
    const size_t px = p.splits > 1 ? (size_t)p.splits * h.M * h.K * 4 : 0;
    const size_t pw = p.splits_w > 1 ? (size_t)p.splits_w * wrows * h.K * 4 : 0;
    p.part = take(px > pw ? px : pw);
    p.total = off;
    return p;
}

namespace {

template <typename T>
PadJob pad_job(const void *in, int64_t ldi, const RowMap &map, int64_t rows, int64_t cols, void *out) {
    constexpr int E = 16 / (int)sizeof(T);
    PadJob j{in, out, map, rows, ldi, cdiv(cols, E) * E, (int)cols, 0};
    while (j.lx < 8 && (1 << j.lx) < cdiv(cols, E)) ++j.lx;
    return j;
}

// X with padded rows, or in position order (sort_x), and W with padded rows,
// those of them that the plan and `x`, `w` ask for
template <typename T>
hipError_t lay_out(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, bool x, bool w, char *ws,
                   hipStream_t s) {
    PadJob j[2];
    int n = 0;
    if (p.pad_x && x) {
        const RowMap map = p.sort_x ? row_map(b.slots, h.M, h.share) : row_map(nullptr, h.M, 1);
        j[n++] = pad_job<T>(b.X, h.ldx, map, p.sort_x ? h.M : h.M / h.share, h.K, ws + p.xpad);
    }
    if (p.pad_w && w) j[n++] = pad_job<T>(b.W, h.ldw, row_map(nullptr, h.M, 1), (h.grouped ? h.G : 1) * h.N, h.K, ws + p.wpad);
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t need = cdiv(j[i].rows, 256 >> j[i].lx);
        if (need > blocks) blocks = need;
    }
    if (blocks > 0)
        k_pad_rows<T><<<dim3((unsigned)(blocks < 65536 ? blocks : 65536), (unsigned)n), 256, 0, s>>>(j[0], j[n - 1]);
    return hipGetLastError();
}

template <typename T>
hipError_t linear_fwd(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, char *ws, hipStream_t s) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t kp = cdiv(h.K, E) * E;
    LinArgs a{};
    a.bias = b.bias, a.R = b.R, a.C = b.Y, a.Z = b.Z;
    a.bf32 = h.bias_f32, a.cf32 = h.ydtype == FK_F32;
    a.ldc = h.ldy, a.ldz = h.ldz, a.ldr = h.ldr;
    a.gsbias = h.N;
    a.offsets = b.offsets;
    a.amap = row_map(b.slots, h.M, h.share);
    a.cmap = row_map(b.slots, h.M, 1);
    a.M = a.rows = h.M, a.N = h.N, a.G = h.grouped ? h.G : 1, a.act = h.act, a.splits = p.splits;
    a.part = (float *)(ws + p.part);
    hipError_t e = hipSuccess;
    if (p.few) {
        a.A = b.X, a.lda = h.ldx, a.B = b.W, a.ldb = h.ldw, a.gsb = h.N * h.ldw, a.ka = a.kb = h.K;
        a.skip = kFewRows;
        e = whole(h.K, h.ldx, h.dtype) && whole(h.K, h.ldw, h.dtype) ? run_few<T, true>(a, s) : run_few<T, false>(a, s);
        if (e != hipSuccess || !p.tiled) return e;
    }
    a.skip = p.few ? kFewRows : 0;
    a.A = b.X, a.lda = h.ldx, a.B = b.W, a.ldb = h.ldw, a.gsb = h.N * h.ldw;
    a.ka = a.kb = kp;
    if ((e = lay_out<T>(h, p, b, true, true, ws, s)) != hipSuccess) return e;
    if (p.pad_x) {
        a.A = ws + p.xpad, a.lda = kp;
        if (p.sort_x) a.amap = row_map(nullptr, h.M, 1);
    }
    if (p.pad_w) a.B = ws + p.wpad, a.ldb = kp, a.gsb = h.N * kp;
    return run_product<T, kFwd>(a, p.tile, s);
}

template <typename T>
hipError_t linear_bwd(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, char *ws, hipStream_t s) {
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t kp = cdiv(h.K, E) * E, np = cdiv(h.N, E) * E;
    const int G = h.grouped ? h.G : 1;
    hipError_t e = hipSuccess;
    LinArgs c{};
    c.offsets = b.offsets, c.cmap = row_map(b.slots, h.M, 1), c.M = h.M, c.N = h.N, c.G = G, c.act = h.act;
    c.Z = (void *)b.Zin, c.ldz = h.ldz;
    c.chunked = on_chunks(b.dY, h.ldy, dtype_size(h.ydtype)) && on_chunks(b.Zin, h.ldz, sizeof(T));
    if ((p.make_dz && (b.dX || b.dW)) || b.db) {
        T *dz = p.make_dz && (b.dX || b.dW) ? (T *)(ws + p.dz) : nullptr;
        float *cs = b.db ? (float *)(ws + p.colsum) : nullptr;
        if (p.grad_tiles > 0) {
            const int64_t grid = p.grad_tiles * cdiv(h.N, 256);
            if (grid > INT32_MAX) return hipErrorInvalidValue;
            k_act_grad<T><<<long_grid(grid), 256, 0, s>>>(c, b.dY, h.ldy, h.ydtype == FK_F32, dz, np, cs, p.grad_tiles);
        }
        if (b.db)
            k_bias_grad<T><<<dim3((unsigned)cdiv(h.N, 16), (unsigned)G), 256, 0, s>>>(c, cs, p.grad_tiles, b.db, h.bias_f32);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const void *X = b.X, *W = b.W;
    int64_t ldx = h.ldx, ldw = h.ldw;
    if ((e = lay_out<T>(h, p, b, b.dW != nullptr, b.dX != nullptr, ws, s)) != hipSuccess) return e;
    if (p.pad_x) X = ws + p.xpad, ldx = kp;
    if (p.pad_w) W = ws + p.wpad, ldw = kp;
    LinArgs a{};
    a.offsets = b.offsets, a.M = h.M, a.G = G, a.act = FK_ACT_NONE, a.part = (float *)(ws + p.part);
    a.A = p.make_dz ? ws + p.dz : b.dY;
    a.lda = p.make_dz ? np : h.ldy;
    a.amap = row_map(p.make_dz ? nullptr : b.slots, h.M, 1);
    if (b.dX) {
        a.B = W, a.ldb = ldw, a.gsb = h.N * ldw, a.bmap = row_map(nullptr, h.M, 1);
        a.C = b.dX, a.ldc = h.lddx, a.cmap = row_map(b.slots, h.M, 1), a.cf32 = sizeof(T) == 4;
        a.rows = h.M, a.N = h.K, a.ka = np, a.kb = h.N, a.splits = p.splits;
        if ((e = run_product<T, kDx>(a, p.tile, s)) != hipSuccess) return e;
    }
    if (b.dW) {
        a.B = X, a.ldb = ldx, a.gsb = 0;
        a.bmap = p.sort_x ? row_map(nullptr, h.M, 1) : row_map(b.slots, h.M, h.share);
        a.C = b.dW, a.ldc = h.K, a.gsc = h.N * h.K, a.cf32 = sizeof(T) == 4;
        a.rows = h.N, a.N = h.K, a.splits = p.splits_w;
        if ((e = run_product<T, kDw>(a, p.tile_w, s)) != hipSuccess) return e;
    }
    return e;
}

}  // namespace

hipError_t launch_linear(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, void *ws, hipStream_t s) {
    switch (h.dtype) {
    case FK_F32: return linear_fwd<float>(h, p, b, (char *)ws, s);
    case FK_BF16: return linear_fwd<__bf16>(h, p, b, (char *)ws, s);
    default: return linear_fwd<_Float16>(h, p, b, (char *)ws, s);
    }
}

hipError_t launch_linear_bwd(const LinearShape &h, const LinearPlan &p, const LinearBufs &b, void *ws, hipStream_t s) {
    switch (h.dtype) {
    case FK_F32: return linear_bwd<float>(h, p, b, (char *)ws, s);
    case FK_BF16: return linear_bwd<__bf16>(h, p, b, (char *)ws, s);
    default: return linear_bwd<_Float16>(h, p, b, (char *)ws, s);
    }
}

}  // namespace fk
