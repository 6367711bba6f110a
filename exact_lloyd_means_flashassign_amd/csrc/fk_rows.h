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

template <typename T>
struct ElemOf;
template <>
struct ElemOf<float> {
    static constexpr int code = FK_F32;
};
template <>
struct ElemOf<__bf16> {
    static constexpr int code = FK_BF16;
};
template <>
struct ElemOf<_Float16> {
    static constexpr int code = FK_F16;
};

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

// Sum over aligned groups of W consecutive lanes (W a power of two up to 64);
// every lane gets it, in the same order in each.
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < W; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
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
