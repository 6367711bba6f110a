// Device helpers of the row-wise operators (layer norm, router, combine) and
// of the products: the element types, 16-byte chunks of them, and sums over a
// team of lanes that shares a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fk.h"

namespace fk {

inline bool known_dtype(int32_t t) { return t == FK_F32 || t == FK_BF16 || t == FK_F16; }
inline size_t dtype_size(int32_t t) { return t == FK_F32 ? 4 : 2; }

// V consecutive elements (V = 1, or as many as 16 bytes hold), kept as they
// lie in memory so that a prefetched chunk costs no more registers than it has
// bytes.
template <typename T, int V>
struct alignas(V * sizeof(T)) Chunk {
    T e[V];
    __device__ __forceinline__ void load(const T *p) { *this = *reinterpret_cast<const Chunk *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Chunk *>(p) = *this; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = (T)0.0f;
    }
};

// V elements of a vector of either its rows' type or fp32
template <typename T, int V>
__device__ __forceinline__ void load_param(const void *p, bool f32, int64_t at, float (&out)[V]) {
    if (f32) {
        constexpr int W = V < 4 ? V : 4;
#pragma unroll
        for (int j = 0; j < V; j += W) {
            Chunk<float, W> c;
            c.load((const float *)p + at + j);
#pragma unroll
            for (int i = 0; i < W; ++i) out[j + i] = c.e[i];
        }
    } else {
        Chunk<T, V> c;
        c.load((const T *)p + at);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = (float)c.e[i];
    }
}

// ---- lane exchanges ----
// Step O of a reduction over aligned groups of lanes, each lane of a group of
// O holding the same value: v of the neighbouring group of O.  Up to groups of
// 16 lanes these are data-parallel moves of the vector ALU (quad permutations and
// mirrors), beyond them permutes through the LDS crossbar, which lanes_reduce
// spares itself by row swaps.
template <int O>
__device__ __forceinline__ uint32_t neighbour(uint32_t v) {
    if constexpr (O == 1) {
        return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);  // quad [1, 0, 3, 2]
    } else if constexpr (O == 2) {
        return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);  // quad [2, 3, 0, 1]
    } else if constexpr (O == 4) {
        return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);  // mirror of 8
    } else if constexpr (O == 8) {
        return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);  // mirror of 16
    } else {
        return __shfl_xor(v, O, 64);
    }
}
template <int O>
__device__ __forceinline__ float neighbour(float v) {
    return __uint_as_float(neighbour<O>(__float_as_uint(v)));
}

// combine(own, neighbour's) over groups of W lanes
template <int W, int O = 1, typename F>
__device__ __forceinline__ float lanes_reduce(float v, F combine) {
    if constexpr (O >= W) {
        return v;
    } else if constexpr (O >= 16) {
        // both operands the same: the first result holds the even rows' values
        // in both rows of a pair, the second the odd rows'
        typedef uint32_t v2u __attribute__((ext_vector_type(2)));
        const uint32_t u = __float_as_uint(v);
        v2u r;
        if constexpr (O == 16) r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane16_swap(u, u, false, false));
        else r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane32_swap(u, u, false, false));
        return lanes_reduce<W, 2 * O>(combine(__uint_as_float(r[0]), __uint_as_float(r[1])), combine);
    } else {
        return lanes_reduce<W, 2 * O>(combine(v, neighbour<O>(v)), combine);
    }
}

// Sum over aligned groups of W consecutive lanes (W a power of two up to 64);
// every lane gets the same.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
    return lanes_reduce<W>(v, [](float a, float b) { return a + b; });
}

// NV sums over a team of TEAM lanes: one wave, or the 256 threads of the
// workgroup (the waves' sums are then added in wave order through LDS; s holds
// 4 * NV floats and is free again after the next call's first barrier, which
// is why calls alternate between two buffers).
template <int TEAM, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float *s) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = lanes_sum<64>(v[i]);
    if constexpr (TEAM > 64) {
        constexpr int WV = TEAM / 64;
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) s[w * NV + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float t = s[i];
#pragma unroll
            for (int j = 1; j < WV; ++j) t += s[j * NV + i];
            v[i] = t;
        }
    }
}

}  // namespace fk
