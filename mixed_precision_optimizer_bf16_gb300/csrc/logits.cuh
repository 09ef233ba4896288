// logits.cuh -- rows of logits, as the kernels over a vocabulary walk them: a CTA's slice of
// a row, its vectors as pairs of FP32 numbers, and their stores.
#pragma once
#include "ops_common.cuh"

namespace bf16ops {

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.f : m; }

// A vector's elements as pairs.
template <class T>
__device__ __forceinline__ void pairs(const uint4 &v, float2 (&f)[Vec<T>::N / 2]) {
    if constexpr (sizeof(T) == 2) {
        f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x)), f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
        f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z)), f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
    } else {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y)), f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // NaN passed over
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Largest element of U vectors (NaN passed over).
template <class T, int U>
__device__ __forceinline__ float largest(const uint4 (&q)[U]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = max_bf16x2(max_bf16x2(q[0].x, q[0].y), max_bf16x2(q[0].z, q[0].w));
#pragma unroll
        for (int u = 1; u < U; ++u) m = max_bf16x2(m, max_bf16x2(max_bf16x2(q[u].x, q[u].y), max_bf16x2(q[u].z, q[u].w)));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
            m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(q[u].x), __uint_as_float(q[u].y))), fmaxf(__uint_as_float(q[u].z), __uint_as_float(q[u].w)));
        return m;
    }
}
// A vector of -inf.
template <class T>
__device__ __forceinline__ uint4 nothing() {
    const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// A row's slice of one CTA: `head` elements before the first 16-byte boundary
// and `tail` after the last whole vector are the first and the last CTA's.
struct Slice {
    uint32_t head, nv, v0, v1;        // whole row: leading elements, vectors; this CTA's vectors [v0, v1)
    uint32_t tail0, lo, hi;           // first trailing element; this CTA's elements are [lo, hi)
};
template <class T>
__device__ __forceinline__ Slice slice_of(const T *row, uint32_t vocab, uint32_t rank, uint32_t ranks, uint32_t log2_ranks) {
    constexpr uint32_t N = Vec<T>::N;
    Slice s;
    const uint32_t off = (uint32_t)((uintptr_t)row & 15u) / (uint32_t)sizeof(T);
    s.head = off ? N - off : 0u;
    if (s.head > vocab) s.head = vocab;
    s.nv = (vocab - s.head) / N;
    s.tail0 = s.head + s.nv * N;
    s.v0 = (uint32_t)(((uint64_t)s.nv * rank) >> log2_ranks);
    s.v1 = (uint32_t)(((uint64_t)s.nv * (rank + 1)) >> log2_ranks);
    s.lo = rank == 0 ? 0u : s.head + s.v0 * N;
    s.hi = rank + 1 == ranks ? vocab : s.head + s.v1 * N;
    return s;
}

// Stores one vector of the gradient: whole where the output row's vectors are
// aligned as the input row's, else element by element.
template <class T>
__device__ __forceinline__ void store_vec(T *out, const float (&g)[Vec<T>::N], bool whole) {
    if (whole) {
        __stcs(reinterpret_cast<uint4 *>(out), Vec<T>::pack(g));
    } else {
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) from_f32(out[i], g[i]);
    }
}

}  // namespace bf16ops
