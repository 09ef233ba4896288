// norm_gate.cu -- the norms before and after a block with its gate and residual
// scale, forward and backward (bf16opt_norm_gate_* of include/bf16opt.h).
//
// Forward: one CTA (or one warp, for short rows) holds a row of x and y in
// registers, so both are read once and r and h written once.  Rows of whole vectors
// come through a ring of shared memory, copied rows ahead.
//
// Backward: a thread owns eight columns and walks down the rows, so the
// weights' and gates' gradients are sums in its registers.  Two norms in a row
// would need two row reductions one after the other; here the second norm's
// sums are linear in the first's results,
//     g = dr + rstd (a - m1 - xhat m2),   a = w dh,
// so eight sums that need neither m1 nor m2 are taken together in one reduction
// and the rest is scalar arithmetic.  A row wider than one CTA's columns is
// split over a cluster, which joins the eight sums through distributed shared
// memory.
//
// Measured on one GB300 (algorithmic bytes over the time; a copy runs at 6.75 TB/s).  Forward, bf16: 32768 rows of
// 2048 102 us, 5.3 TB/s; 4096 of 14336 125 us, 3.8 TB/s; those with an FP32 stream and a gate 167 us,
// 4.2 TB/s.  Backward: 32768 of 2048 181 us, 4.4 TB/s; 4096 of 14336 182 us, 3.9 TB/s; 8192 of 2048 with biases and a
// gate for each sequence 68 us, 3.0 TB/s.  What bounds a wide row is its own chain -- loads, reductions one after the other,
// stores -- with one or two CTAs in an SM (warps active 22 %, issue slots 33 % forward, 51 % backward).  The backward
// kernels with two runs a thread spill 76 to 116 bytes under their 128 registers; they would not at 144, which
// 448 threads could have where one CTA is all that an SM holds (not measured).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace bf16ops {
namespace {

struct Norm {
    int kind;             // BF16OPT_NORM_*
    const void *weight, *bias;
};

struct Args {
    uint64_t rows;
    uint32_t hidden;
    int weight_type;
    Norm pre, post;
    int gate_act;
    uint64_t gate_rows, rows_per_gate;
    const void *gate;
    float residual_scale, branch_scale, eps;
};

// ------------------------------------------------------- eight elements of a row
// VEC: element i of slot v of thread t is (v * threads + t) * 8 + i, moved as
// 16-byte vectors; else (v * 8 + i) * threads + t, moved one by one (rows of
// any length and alignment).

template <bool VEC>
__device__ __forceinline__ uint32_t column(uint32_t slot, uint32_t threads, uint32_t t, uint32_t i) {
    return VEC ? (slot * threads + t) * 8 + i : (slot * 8 + i) * threads + t;
}

template <bool VEC, class T>
__device__ __forceinline__ void load8(const T *row, uint32_t n, uint32_t slot, uint32_t threads, uint32_t t, float (&f)[8]) {
    if constexpr (VEC) {
        const uint32_t c = column<true>(slot, threads, t, 0);
        if (c < n) {
            if constexpr (sizeof(T) == 2) {
                Vec<T>::unpack(__ldcs(reinterpret_cast<const uint4 *>(row + c)), f);
            } else {
                const float4 a = __ldcs(reinterpret_cast<const float4 *>(row + c)), b = __ldcs(reinterpret_cast<const float4 *>(row + c) + 1);
                f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = column<false>(slot, threads, t, i);
            f[i] = c < n ? to_f32(row[c]) : 0.f;
        }
    }
}

template <bool VEC, class T>
__device__ __forceinline__ void store8(T *row, uint32_t n, uint32_t slot, uint32_t threads, uint32_t t, const float (&f)[8]) {
    if constexpr (VEC) {
        const uint32_t c = column<true>(slot, threads, t, 0);
        if (c < n) {
            if constexpr (sizeof(T) == 2) {
                __stcs(reinterpret_cast<uint4 *>(row + c), Vec<T>::pack(f));
            } else {
                __stcs(reinterpret_cast<float4 *>(row + c), make_float4(f[0], f[1], f[2], f[3]));
                __stcs(reinterpret_cast<float4 *>(row + c) + 1, make_float4(f[4], f[5], f[6], f[7]));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = column<false>(slot, threads, t, i);
            if (c < n) from_f32(row[c], f[i]);
        }
    }
}

// Weights: read again and again, so kept in L1.  Beyond the row 0, also where there are none: a norm that
// subtracts a mean leaves nothing there then, and the next norm's mean is the row's alone.
template <bool VEC>
__device__ __forceinline__ void load8_weight(const void *w, int type, uint32_t n, uint32_t slot, uint32_t threads, uint32_t t,
                                             float none, float (&f)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = column<VEC>(slot, threads, t, VEC ? 0 : i) < n ? none : 0.f;
        return;
    }
    if constexpr (VEC) {
        const uint32_t c = column<true>(slot, threads, t, 0);
        if (c < n) {
            if (type == BF16OPT_TYPE_BF16) {
                Vec<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(w) + c)), f);
            } else {
                const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(w) + c);
                const float4 a = __ldg(p), b = __ldg(p + 1);
                f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = column<false>(slot, threads, t, i);
            f[i] = c < n ? load_typed(w, type, c) : 0.f;
        }
    }
}

__device__ __forceinline__ float sigmoid(float x) {
    float y;   // the reciprocal to one unit in the last place
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + ex2(-x * kLog2e)));
    return y;
}

// Eight columns of a row as four pairs.
struct Cols {
    float2 v[4];
};
template <class T>
__device__ __forceinline__ Cols unpack8(const uint4 *p, uint32_t stride) {
    Cols c;
    const uint4 a = p[0];
    if constexpr (sizeof(T) == 2) {
        c.v[0] = make_float2(bf16_lo(a.x), bf16_hi(a.x)), c.v[1] = make_float2(bf16_lo(a.y), bf16_hi(a.y));
        c.v[2] = make_float2(bf16_lo(a.z), bf16_hi(a.z)), c.v[3] = make_float2(bf16_lo(a.w), bf16_hi(a.w));
    } else {
        const uint4 b = p[stride];
        c.v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y)), c.v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
        c.v[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y)), c.v[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
    return c;
}
// The same from a place between two 16-byte boundaries: p holds the vectors from the boundary before on, one
// more than the columns fill, `mis` is how many bytes of the first come before the columns.
template <class T>
__device__ __forceinline__ Cols unpack8_shifted(const uint4 *p, uint32_t stride, uint32_t mis) {
    constexpr int NW = sizeof(T) == 2 ? 8 : 12, N = sizeof(T) == 2 ? 5 : 8;   // words there, words needed
    uint32_t w[NW];
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) {
        const uint4 q = p[i * stride];
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i <= N; ++i) w[i] = mis & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = mis & 4 ? w[i + 1] : w[i];
    Cols c;
    if constexpr (sizeof(T) == 2) {
        const uint32_t pick = mis & 2 ? 0x5432u : 0x3210u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __byte_perm(w[i], w[i + 1], pick);
            c.v[i] = make_float2(bf16_lo(x), bf16_hi(x));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) c.v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    return c;
}
__device__ __forceinline__ Cols all8(float x) {
    Cols c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.v[i] = both(x);
    return c;
}
__device__ __forceinline__ Cols cols_of(const float (&f)[8]) {
    Cols c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    return c;
}
// Eight columns from `c` on of a row of n, one by one, 0 beyond the row.
template <class T>
__device__ __forceinline__ Cols load_cols(const T *row, uint32_t c, uint32_t n) {
    float f[8];
    if (c + 8 <= n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_f32(row[c + i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < n ? to_f32(row[c + i]) : 0.f;
    }
    return cols_of(f);
}
// And stored.  VEC: whole vectors, all of them there or none; else one by one.
template <bool VEC, class T>
__device__ __forceinline__ void store_cols(T *row, uint32_t c, uint32_t n, const Cols &x) {
    const float f[8] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y, x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
    if (VEC) {
        if (c >= n) return;
        if constexpr (sizeof(T) == 2) {
            __stcs(reinterpret_cast<uint4 *>(row + c), Vec<T>::pack(f));
        } else {
            __stcs(reinterpret_cast<float4 *>(row + c), make_float4(f[0], f[1], f[2], f[3]));
            __stcs(reinterpret_cast<float4 *>(row + c) + 1, make_float4(f[4], f[5], f[6], f[7]));
        }
    } else if (c + 8 <= n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) from_f32(row[c + i], f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) from_f32(row[c + i], f[i]);
    }
}
// Eight columns of a row on a 16-byte boundary; VEC: all of them there or none.
template <bool VEC, class T>
__device__ __forceinline__ void store_cols_ended(T *row, uint32_t c, uint32_t n, const Cols &x) {
    if (VEC || c + 8 <= n) store_cols<true>(row, c, n, x);
    else store_cols<false>(row, c, n, x);
}
// Eight columns from c on, c a multiple of eight that grows by eight from lane to lane, of a row that begins
// between two 16-byte boundaries: a lane stores the vectors that its columns begin in, together with the lane
// before, whose last columns it gets by a shuffle; the columns at a warp's and the row's ends go one by one.
// Every lane of the warp calls it.
template <class T>
__device__ __forceinline__ void store_cols_shifted(T *row, uint32_t c, uint32_t n, const Cols &x, uint32_t lane) {
    constexpr int NW = sizeof(T) == 2 ? 4 : 8, BEFORE = sizeof(T) == 2 ? 4 : 3;
    const float f[8] = {x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y, x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y};
    uint32_t w[BEFORE + NW + 1];   // the last words of the lane before, this lane's
    if constexpr (sizeof(T) == 2) {
        const uint4 q = Vec<T>::pack(f);
        w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[3 + i] = __float_as_uint(f[i]);
    }
    w[BEFORE + NW] = 0u;
#pragma unroll
    for (int i = 0; i < BEFORE; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[NW + i], 1);
    const uint32_t mis = (uint32_t)(uintptr_t)row & 15u, ends = 8 - mis / (uint32_t)sizeof(T);   // columns [ends, 8) are the next lane's to store
    const bool mine = lane != 0 && c + 8 <= n, next = lane != 31 && c + 16 <= n;
    if (!mine || !next) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n && !(i < (int)ends ? mine : next)) from_f32(row[c + i], f[i]);
    }
    const uint32_t back = BEFORE * 4 - mis;   // where in w the vectors begin, in bytes
    if constexpr (sizeof(T) == 2) {           // 2 .. 14: mis is not 0
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = back & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = back & 4 ? w[i + 1] : w[i];
        const uint32_t pick = back & 2 ? 0x5432u : 0x3210u;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], w[i + 1], pick);
    } else {                                  // 0, 4, 8
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = back & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = back & 4 ? w[i + 1] : w[i];
    }
    if (mine) {
        uint4 *to = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(row + c) - mis);
        __stcs(to, make_uint4(w[0], w[1], w[2], w[3]));
        if constexpr (sizeof(T) == 4) __stcs(to + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}
__device__ __forceinline__ float2 sigmoid2(float2 x) { return make_float2(sigmoid(x.x), sigmoid(x.y)); }

// ------------------------------------------------------------------------ forward

// Sum over the CTA's threads of one row (a warp, or the whole CTA); the two
// halves of `buf` alternate, so one barrier per sum is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *buf, uint32_t &turn) {
    v = warp_sum(v);
    if constexpr (WARP) {
        return v;
    } else {
        float *b = buf + (turn & 1) * 32;
        ++turn;
        if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
        __syncthreads();
        float s = 0.f;
        for (uint32_t i = 0; i < blockDim.x / 32; ++i) s += b[i];
        return s;
    }
}

// Mean and 1 / sqrt(.. + eps) of the row in v; elements beyond the row are 0.
// Two sums one after the other (mean, then squares of the rest): a variance
// from the sums of v and v^2 would cancel where the mean is large.
template <bool VEC, bool WARP, int NV>
__device__ __forceinline__ void moments(const float (&v)[NV][8], int kind, uint32_t n, float eps, uint32_t threads, uint32_t t,
                                        float *buf, uint32_t &turn, float &mean, float &rstd) {
    mean = 0.f;
    if (kind == BF16OPT_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[k][i];
        mean = row_sum<WARP>(s, buf, turn) / (float)n;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = column<VEC>(k, threads, t, i) < n ? v[k][i] - mean : 0.f;
            q = fmaf(d, d, q);
        }
    rstd = 1.f / sqrtf(row_sum<WARP>(q, buf, turn) / (float)n + eps);
}

template <class TB, class TS, bool VEC, bool WARP, int NV>
__global__ void __launch_bounds__(WARP ? 128 : 512)
k_norm_forward(const Args a, const TS *x, const TB *y, TS *r, TB *h, float *stats, uint64_t row0) {
    __shared__ float buf[64];
    const uint32_t threads = WARP ? 32u : blockDim.x, t = WARP ? threadIdx.x & 31u : threadIdx.x;
    const uint32_t n = a.hidden;
    uint32_t turn = 0;
    pdl_enter();
    const uint64_t row = row0 + (WARP ? (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x);
    if (row >= a.rows) return;   // whole warps (WARP) or none
    float u[NV][8], v[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) load8<VEC>(y + row * n, n, k, threads, t, u[k]);
#pragma unroll
    for (int k = 0; k < NV; ++k) load8<VEC>(x + row * n, n, k, threads, t, v[k]);
    float mean = 0.f, rstd = 0.f;
    if (a.post.kind != BF16OPT_NORM_NONE) {
        moments<VEC, WARP, NV>(u, a.post.kind, n, a.eps, threads, t, buf, turn, mean, rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8], b[8];
            load8_weight<VEC>(a.post.weight, a.weight_type, n, k, threads, t, 1.f, w);
            load8_weight<VEC>(a.post.bias, a.weight_type, n, k, threads, t, 0.f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[k][i] = fmaf((u[k][i] - mean) * rstd, w[i], b[i]);
        }
    }
    if (stats && t == 0) stats[4 * row + 2] = mean, stats[4 * row + 3] = rstd;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (a.gate) {
            float g[8];
            load8<VEC>(reinterpret_cast<const TB *>(a.gate) + row / a.rows_per_gate * n, n, k, threads, t, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[k][i] *= a.gate_act == BF16OPT_GATE_SIGMOID ? sigmoid(g[i]) : g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = fmaf(a.residual_scale, v[k][i], a.branch_scale * u[k][i]);
        store8<VEC>(r + row * n, n, k, threads, t, v[k]);
    }
    mean = rstd = 0.f;
    if (a.pre.kind != BF16OPT_NORM_NONE) {
        moments<VEC, WARP, NV>(v, a.pre.kind, n, a.eps, threads, t, buf, turn, mean, rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float w[8], b[8];
            load8_weight<VEC>(a.pre.weight, a.weight_type, n, k, threads, t, 1.f, w);
            load8_weight<VEC>(a.pre.bias, a.weight_type, n, k, threads, t, 0.f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = fmaf((v[k][i] - mean) * rstd, w[i], b[i]);
            store8<VEC>(h + row * n, n, k, threads, t, w);
        }
    }
    if (stats && t == 0) stats[4 * row] = mean, stats[4 * row + 1] = rstd;
}

// Rows of whole vectors: a CTA walks down its rows, which come through a ring in
// shared memory whose slots belong to one thread each, filled by asynchronous
// copies `depth` rows ahead: with a row's loads, its two to four reductions one after the other
// and its stores all in one CTA after the other, an SM that holds one wide row
// moved 4.1 TB/s.  A thread has V runs of eight columns, `threads` runs apart.
template <class TB, class TS, bool GATE, int V>
__global__ void __launch_bounds__(V == 4 ? 512 : 384, V == 4 ? 1 : 2) k_norm_forward_ring(const Args a, const TS *x, const TB *y, TS *r, TB *h, float *stats, uint32_t depth) {
    constexpr int UB = sizeof(TB) / 2, US = sizeof(TS) / 2, UNITS = (GATE ? 2 : 1) * UB + US;   // y, x, [gate]
    extern __shared__ __align__(128) unsigned char ring_raw[];
    __shared__ float buf[64];
    const uint32_t threads = blockDim.x, t = threadIdx.x, n = a.hidden;
    auto col = [&](int v) { return (v * threads + t) * 8; };
    uint4 *ring = reinterpret_cast<uint4 *>(ring_raw) + t;   // [slot][run][unit][thread]
    const uint32_t slot_units = threads * UNITS * V;
    uint32_t turn = 0;
    pdl_enter();
    const uint64_t row0 = team_row(a.rows, gridDim.x, blockIdx.x), row1 = team_row(a.rows, gridDim.x, blockIdx.x + 1);
    uint64_t copy_row = row0, gate_row = GATE ? row0 / a.rows_per_gate : 0, gate_left = GATE ? (gate_row + 1) * a.rows_per_gate - row0 : 0;
    uint32_t copy_slot = 0;
    auto fill = [&]() {
        if (copy_row < row1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (col(v) < n) {
                    uint4 *to = ring + copy_slot * slot_units + v * UNITS * threads;
                    const uint64_t o = copy_row * n + col(v);
#pragma unroll
                    for (int i = 0; i < UB; ++i) copy_async16(to + i * threads, reinterpret_cast<const uint4 *>(y + o) + i);
#pragma unroll
                    for (int i = 0; i < US; ++i) copy_async16(to + (UB + i) * threads, reinterpret_cast<const uint4 *>(x + o) + i);
                    if (GATE) {
                        const TB *g = reinterpret_cast<const TB *>(a.gate) + gate_row * n + col(v);
#pragma unroll
                        for (int i = 0; i < UB; ++i) copy_async16(to + (UB + US + i) * threads, reinterpret_cast<const uint4 *>(g) + i);
                    }
                }
            }
        }
        copy_commit();
        ++copy_row;
        if (GATE && --gate_left == 0) ++gate_row, gate_left = a.rows_per_gate;
        copy_slot = copy_slot + 1 == depth ? 0 : copy_slot + 1;
    };
    for (uint32_t s = 0; s < depth; ++s) fill();
    // The first 16 bytes of a weight's or bias's run: all of a bf16 one, half of an FP32 one. The weights'
    // are asked for before the reduction that comes before their use: they come from L2 where
    // the ring leaves L1 no room for them.
    auto first16 = [&](const void *w, int v) {
        return __ldg(reinterpret_cast<const uint4 *>((const char *)w + (size_t)col(v) * (a.weight_type == BF16OPT_TYPE_BF16 ? 2 : 4)));
    };
    auto weight = [&](const void *w, int v, const uint4 &first) {
        uint4 q[2] = {first, first};
        if (a.weight_type == BF16OPT_TYPE_BF16) return unpack8<__nv_bfloat16>(q, 0);
        q[1] = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(w) + col(v)) + 1);
        return unpack8<float>(q, 1);
    };
    uint4 ahead[V];
    auto ask = [&](const Norm &norm) {
        if (norm.weight)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (col(v) < n) ahead[v] = first16(norm.weight, v);
    };
    const float inv_n = 1.f / (float)n;
    // Mean and 1/deviation of the row in u, as moments() but by pairs; runs beyond the row stay out.
    auto moments2 = [&](const Cols(&u)[V], int kind, float &mean, float &rstd) {
        mean = 0.f;
        if (kind == BF16OPT_NORM_LAYER) {
            float2 s = both(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) s = add2(s, u[v].v[i]);
            mean = row_sum<false>(s.x + s.y, buf, turn) * inv_n;
        }
        float2 q = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (col(v) < n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 d = add2(u[v].v[i], both(-mean));
                    q = fma2(d, d, q);
                }
        rstd = 1.f / sqrtf(row_sum<false>(q.x + q.y, buf, turn) * inv_n + a.eps);
    };
    // (u - mean) rstd weight + bias
    auto normed = [&](Cols u, const Norm &norm, float mean, float rstd, int v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u.v[i] = mul2(add2(u.v[i], both(-mean)), both(rstd));
        if (norm.weight) {
            const Cols w = weight(norm.weight, v, ahead[v]);
#pragma unroll
            for (int i = 0; i < 4; ++i) u.v[i] = mul2(u.v[i], w.v[i]);
        }
        if (norm.bias) {
            const Cols b = weight(norm.bias, v, first16(norm.bias, v));
#pragma unroll
            for (int i = 0; i < 4; ++i) u.v[i] = add2(u.v[i], b.v[i]);
        }
        return u;
    };
    uint32_t slot = 0;
    const float2 rs = both(a.residual_scale), bs = both(a.branch_scale);
    for (uint64_t row = row0; row < row1; ++row) {
        copy_wait_for(depth - 1);
        const uint4 *from = ring + slot * slot_units;
        Cols u[V];
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = col(v) < n ? unpack8<TB>(from + v * UNITS * threads, threads) : all8(0.f);
        float mean = 0.f, rstd = 0.f;
        const bool post = a.post.kind != BF16OPT_NORM_NONE;
        if (post) {
            ask(a.post);
            moments2(u, a.post.kind, mean, rstd);
        }
        if (stats && t == 0) stats[4 * row + 2] = mean, stats[4 * row + 3] = rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (col(v) < n) {   // else it stays 0
                if (post) u[v] = normed(u[v], a.post, mean, rstd, v);
                if (GATE) {
                    const Cols g = unpack8<TB>(from + (v * UNITS + UB + US) * threads, threads);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        u[v].v[i] = mul2(u[v].v[i], a.gate_act == BF16OPT_GATE_SIGMOID ? sigmoid2(g.v[i]) : g.v[i]);
                }
                const Cols in = unpack8<TS>(from + (v * UNITS + UB) * threads, threads);
#pragma unroll
                for (int i = 0; i < 4; ++i) u[v].v[i] = fma2(rs, in.v[i], mul2(bs, u[v].v[i]));
                store_cols<true>(r + row * n, col(v), n, u[v]);
            }
        }
        fill();   // the row's inputs are read
        slot = slot + 1 == depth ? 0 : slot + 1;
        mean = rstd = 0.f;
        if (a.pre.kind != BF16OPT_NORM_NONE) {
            ask(a.pre);
            moments2(u, a.pre.kind, mean, rstd);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (col(v) < n) store_cols<true>(h + row * n, col(v), n, normed(u[v], a.pre, mean, rstd, v));
        }
        if (stats && t == 0) stats[4 * row] = mean, stats[4 * row + 1] = rstd;
    }
    pdl_leave();
}

// ----------------------------------------------------------------------- backward

// 16-byte units of eight columns in the ring: one more where they lie between boundaries.
template <class T, bool VEC>
__host__ __device__ constexpr int units() {
    return (int)sizeof(T) / 2 + (VEC ? 0 : 1);
}
// A thread's eight columns into its units, `stride` apart: columns c on of the row's n from element `off` on
// of a tensor of `size`.  Not VEC: the vectors from the boundary before to the one after, the
// columns' own elements alone at the tensor's ends.
template <bool VEC, class E>
__device__ __forceinline__ void copy_run(uint4 *to, uint32_t stride, const E *tensor, uint64_t off, uint32_t c, uint32_t n, uint64_t size) {
    const uintptr_t from = VEC ? (uintptr_t)(tensor + off + c) : (uintptr_t)(tensor + off + c) & ~(uintptr_t)15;
    if (VEC || (off >= 16 && off + n + 32 <= size)) {
#pragma unroll
        for (int i = 0; i < units<E, VEC>(); ++i) copy_async16(to + i * stride, reinterpret_cast<const uint4 *>(from) + i);
    } else {
        constexpr uint32_t PER = 16 / sizeof(E);
        for (uint32_t e = 0; e < units<E, VEC>() * PER; ++e) {
            const uintptr_t p = from + e * sizeof(E);
            if (p >= (uintptr_t)tensor && p < (uintptr_t)(tensor + size))
                reinterpret_cast<E *>(to + e / PER * stride)[e % PER] = *reinterpret_cast<const E *>(p);
        }
    }
}
// And out of them again; 0 beyond the row.
__device__ __forceinline__ void end_row(Cols &x, uint32_t c, uint32_t n) {
    if (c + 8 <= n) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (c + 2 * i >= n) x.v[i].x = 0.f;
        if (c + 2 * i + 1 >= n) x.v[i].y = 0.f;
    }
}
template <bool VEC, class E>
__device__ __forceinline__ Cols read_run(const uint4 *from, uint32_t stride, const E *tensor, uint64_t off, uint32_t c, uint32_t n) {
    if constexpr (VEC) return unpack8<E>(from, stride);
    Cols x = unpack8_shifted<E>(from, stride, (uint32_t)(uintptr_t)(tensor + off) & 15u);
    end_row(x, c, n);
    return x;
}
template <bool VEC, class E>
__device__ __forceinline__ void store_run(E *row, uint32_t c, uint32_t n, const Cols &x, uint32_t lane) {   // by the whole warp
    if (VEC || ((uintptr_t)row & 15u) == 0) store_cols_ended<VEC>(row, c, n, x);
    else store_cols_shifted(row, c, n, x, lane);
}

// Threads of a CTA at most, and with them the columns: 448 threads of 128 registers, each
// with one or two runs of eight columns.  With 8 columns a thread, what a row costs a warp
// apart from its columns (the two reductions, addresses, copies) was as much as the
// columns: 608 instructions a row of 8, 282 us on 4096 x 14336, against 217 us with 16.
constexpr int kBackThreads = 448;
constexpr int kSums = 8;         // per row

struct BackArgs {
    const void *dr, *dh, *r, *y;
    const float *stats;
    void *dx, *dy, *dgate;
    // FP32 partial sums: [teams][4][hidden] of the weights' gradients, and
    // [2 teams][hidden] of the gates' that straddle teams
    float *part, *gate_part;
    uint32_t teams;
    uint32_t want;         // bits: the weights' gradients asked for, in the order of part
    bool shared_gate;      // rows share gate rows and dgate is wanted
};

// Sum of eight values over a warp: each step a lane keeps half of the values
// and hands the other half over, so it costs 9 shuffles, not 40.  Lane l ends up
// with the sum of value lane_value(l & 7): its bits reversed.
__device__ __forceinline__ float warp_sum8(const float (&s)[8], uint32_t lane) {
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 1;
        const float give = up ? s[i] : s[i + 4], keep = up ? s[i + 4] : s[i];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 2;
        const float give = up ? a[i] : a[i + 2], keep = up ? a[i + 2] : a[i];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    {
        const bool up = lane & 4;
        const float give = up ? b[0] : b[1], keep = up ? b[1] : b[0];
        c = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
    c += __shfl_xor_sync(0xffffffffu, c, 8);
    c += __shfl_xor_sync(0xffffffffu, c, 16);
    return c;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t lane) { return (lane & 1) * 4 + (lane & 2) + ((lane & 4) >> 2); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 16-byte units of eight columns of a row that a thread keeps in the ring: y, dh, [gate] of the
// branch's type, r, dr of the stream's; not VEC: the eight columns lie between boundaries, in one more.
template <class TB, class TS, bool VEC, int GATE>
__host__ __device__ constexpr int ring_units() {
    return (GATE == 1 ? 3 : 2) * units<TB, VEC>() + 2 * units<TS, VEC>();
}

// A team (a CTA, or a cluster that shares the columns) walks down its rows in two
// overlapped steps: the sums of row k + 1 are taken and published while those of
// row k are still on their way, then row k's outputs are written.  The rows
// come through a ring in shared memory whose slots belong to one thread each, filled
// by asynchronous copies `depth` rows ahead.  A thread has V runs of eight columns,
// `threads` runs apart.  VEC: rows of whole 16-byte vectors; else a run lies between
// boundaries: it is copied with one more vector, and shifted into place when it is read
// (element by element, twice from L1: 8192 x 4097 bf16 585 us, so 282 us).
// GATE: 0 none; 1 a row of it comes with each row; 2 many rows share one (kGateRows at
// least): its values are in w2, and since they are the same for all those rows, P = sum g yhat
// and Q = sum g down the rows give all that depends on it when the rows end:
//     dgate = act' (weight P + bias Q),  dweight += act P,  dbias += act Q.
// There the row after the last is published only when the gate has changed.
constexpr uint64_t kGateRows = 8;
template <class TB, class TS, bool VEC, int GATE, int V>
__global__ void __launch_bounds__(kBackThreads, 1) k_norm_backward(const Args a, const BackArgs q, uint32_t depth) {
    constexpr int UNITS = ring_units<TB, TS, VEC, GATE>(), UB = units<TB, VEC>(), US = units<TS, VEC>();
    extern __shared__ __align__(128) unsigned char ring_raw[];
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t threads = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = threads / 32;
    const uint32_t team = blockIdx.x / ranks;
    // this CTA's columns: [c0, c0 + n); this thread's runs begin at col(0), col(1) ...
    const uint32_t c0 = rank * threads * 8 * V;
    const uint32_t n = c0 < a.hidden ? min(a.hidden - c0, threads * 8 * V) : 0u;
    auto col = [&](int v) { return (v * threads + t) * 8; };
    const float inv_h = 1.f / (float)a.hidden;
    const bool pre = a.pre.kind != BF16OPT_NORM_NONE && q.dh, post = a.post.kind != BF16OPT_NORM_NONE;
    const bool pre_layer = a.pre.kind == BF16OPT_NORM_LAYER, post_layer = a.post.kind == BF16OPT_NORM_LAYER;
    pdl_enter();
    if (ranks > 1) cluster.sync();

    const uint64_t row0 = team_row(a.rows, q.teams, team), row1 = team_row(a.rows, q.teams, team + 1);
    uint4 *ring = reinterpret_cast<uint4 *>(ring_raw) + t;   // [slot][run][unit][thread]
    const uint32_t slot_units = threads * UNITS * V;
    // Sums of a row, [rank, warp][kSums], three rows deep: a CTA may still read one row's
    // after it has arrived for the next, when another sets out with the one after that.
    float *sm_sums = reinterpret_cast<float *>(ring_raw + (size_t)depth * slot_units * 16);
    const uint32_t entries = ranks * warps;
    uint32_t sums_at = 0;   // of the row that is worked on
    auto sums_next = [&](uint32_t at) { return at == 2 * entries * kSums ? 0u : at + entries * kSums; };

    // Which gate row a row has, and how many rows it has it for still: one division at the
    // start. One for the copies, one for the rows as they are worked on.
    struct GateRow {
        uint64_t row, left;
    };
    GateRow copy_gate = {0, 0};
    if (GATE) copy_gate.row = row0 / a.rows_per_gate, copy_gate.left = (copy_gate.row + 1) * a.rows_per_gate - row0;
    GateRow gate = copy_gate;
    auto gate_next = [&](GateRow &g) {
        if (GATE && --g.left == 0) ++g.row, g.left = a.rows_per_gate;
    };

    uint64_t copy_row = row0;
    uint32_t copy_slot = 0;
    // Copies the next row into its slot; missing inputs stay the zeros they are made below.
    auto fill = [&]() {
        if (copy_row < row1) {
            const uint64_t o = copy_row * a.hidden + c0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (col(v) >= n) break;
                uint4 *to = ring + copy_slot * slot_units + v * UNITS * threads;
                auto put = [&](int at, const auto *base, uint64_t off, uint64_t rows) {
                    copy_run<VEC>(to + at * threads, threads, base, off, col(v), n, rows * a.hidden);
                };
                put(0, reinterpret_cast<const TB *>(q.y), o, a.rows);
                if (pre) {
                    put(UB, reinterpret_cast<const TB *>(q.dh), o, a.rows);
                    put(2 * UB, reinterpret_cast<const TS *>(q.r), o, a.rows);
                }
                if (q.dr) put(2 * UB + US, reinterpret_cast<const TS *>(q.dr), o, a.rows);
                if (GATE == 1) put(2 * UB + 2 * US, reinterpret_cast<const TB *>(a.gate), copy_gate.row * a.hidden + c0, a.gate_rows);
            }
        }
        copy_commit();
        ++copy_row;
        gate_next(copy_gate);
        copy_slot = copy_slot + 1 == depth ? 0 : copy_slot + 1;
    };
    for (uint32_t s = 0; s < depth; ++s)   // what no copy fills
#pragma unroll
        for (int v = 0; v < V; ++v)
            for (int i = 0; i < UNITS; ++i)
                if (col(v) >= n || (!pre && i >= UB && i < 2 * UB + US) || (!q.dr && i >= 2 * UB + US && i < 2 * UB + 2 * US))
                    ring[s * slot_units + (v * UNITS + i) * threads] = make_uint4(0, 0, 0, 0);
    for (uint32_t s = 0; s < depth; ++s) fill();
    struct Run {
        Cols y, dh, r, dr, gate;
    };
    auto load_run = [&](uint64_t row, uint32_t slot, const GateRow &g, int v) {
        Run w;
        const uint4 *p = ring + slot * slot_units + v * UNITS * threads;
        auto get = [&](int at, const auto *base, uint64_t off) { return read_run<VEC>(p + at * threads, threads, base, off, col(v), n); };
        const uint64_t o = row * a.hidden + c0;
        w.y = get(0, reinterpret_cast<const TB *>(q.y), o);
        w.dh = get(UB, reinterpret_cast<const TB *>(q.dh), o);
        w.r = get(2 * UB, reinterpret_cast<const TS *>(q.r), o);
        w.dr = get(2 * UB + US, reinterpret_cast<const TS *>(q.dr), o);
        if constexpr (GATE == 1) w.gate = get(2 * UB + 2 * US, reinterpret_cast<const TB *>(a.gate), g.row * a.hidden + c0);
        return w;
    };
    // Statistics of a row: mean and 1/deviation of r and of y; of a norm that is not there 0 and 1.
    auto stats_of = [&](uint64_t row) {
        float4 s = make_float4(0.f, 1.f, 0.f, 1.f);
        if (row < row1) {
            if (pre) s.x = q.stats[4 * row], s.y = q.stats[4 * row + 1];
            if (post) s.z = q.stats[4 * row + 2], s.w = q.stats[4 * row + 3];
        }
        return s;
    };

    // weights: 0 beyond the row, so that what is there counts for nothing; the post-norm's
    // with the branch's scale in it
    auto weights = [&](const void *w, float none, float scale, int v) {
        Cols c = all8(0.f);
        if (col(v) >= n) return c;
        if (!w) c = all8(none);
        else if (VEC && a.weight_type == BF16OPT_TYPE_BF16)
            c = unpack8<__nv_bfloat16>(reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(w) + c0 + col(v)), 1);
        else if (VEC)
            c = unpack8<float>(reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(w) + c0 + col(v)), 1);
        else if (a.weight_type == BF16OPT_TYPE_BF16)
            c = load_cols(reinterpret_cast<const __nv_bfloat16 *>(w) + c0, col(v), n);
        else
            c = load_cols(reinterpret_cast<const float *>(w) + c0, col(v), n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c.v[i] = mul2(c.v[i], both(scale));
            if (!VEC && !w) {   // the last run may be part of the row only
                if (col(v) + 2 * i >= n) c.v[i].x = 0.f;
                if (col(v) + 2 * i + 1 >= n) c.v[i].y = 0.f;
            }
        }
        return c;
    };
    Cols w1[V], w2[V], b2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w1[v] = weights(a.pre.weight, 1.f, 1.f, v);
        w2[v] = weights(a.post.weight, 1.f, a.branch_scale, v);
        if (GATE == 1) b2[v] = weights(a.post.bias, 0.f, a.branch_scale, v);
    }

    // sums down the rows; of the post-norm's gradients without the branch's scale, which comes at the end
    Cols dw1[V], db1[V], dw2[V], db2[V], dg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dw1[v] = db1[v] = dw2[v] = db2[v] = dg[v] = all8(0.f);
    const float2 rs = both(a.residual_scale);

    // GATE 2: the gate row's values into w2, and what its rows came to
    auto gate_cols = [&](int v) {
        const TB *g = reinterpret_cast<const TB *>(a.gate) + gate.row * a.hidden + c0;
        if (!VEC) return load_cols(g, col(v), n);
        return col(v) < n ? unpack8<TB>(reinterpret_cast<const uint4 *>(g + col(v)), 1) : all8(0.f);
    };
    auto take_gate = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            w2[v] = weights(a.post.weight, 1.f, a.branch_scale, v);
            const Cols g = gate_cols(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) w2[v].v[i] = mul2(w2[v].v[i], a.gate_act == BF16OPT_GATE_SIGMOID ? sigmoid2(g.v[i]) : g.v[i]);
        }
    };
    bool gates_before = false;
    auto end_gate = [&](bool whole, bool last_of_team) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols g = gate_cols(v), w = weights(a.post.weight, 1.f, a.branch_scale, v), b = weights(a.post.bias, 0.f, a.branch_scale, v);
            Cols d;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 act = g.v[i], slope = both(1.f);
                if (a.gate_act == BF16OPT_GATE_SIGMOID) {
                    act = sigmoid2(act);
                    slope = mul2(act, make_float2(1.f - act.x, 1.f - act.y));
                }
                d.v[i] = mul2(slope, fma2(w.v[i], dw2[v].v[i], mul2(b.v[i], db2[v].v[i])));
                dw2[v].v[i] = mul2(act, dw2[v].v[i]), db2[v].v[i] = mul2(act, db2[v].v[i]);
            }
            if (q.dgate) {
                if (whole) store_cols<VEC>(reinterpret_cast<TB *>(q.dgate) + gate.row * a.hidden + c0, col(v), n, d);
                else store_cols<VEC>(q.gate_part + (size_t)(2 * team + (gate.row * a.rows_per_gate > row0 ? 1 : 0)) * a.hidden + c0, col(v), n, d);
            }
            // the weights' sums over the gates so far are kept where the partial sums go
            float *p = q.part + (size_t)team * 4 * a.hidden + c0;
            if (gates_before) {
                auto kept = [&](const float *f) {
                    if (!VEC) return load_cols(f, col(v), n);
                    return col(v) < n ? unpack8<float>(reinterpret_cast<const uint4 *>(f + col(v)), 1) : all8(0.f);
                };
                const Cols w0 = kept(p + 2 * (size_t)a.hidden), b0 = kept(p + 3 * (size_t)a.hidden);
#pragma unroll
                for (int i = 0; i < 4; ++i) dw2[v].v[i] = add2(w0.v[i], dw2[v].v[i]), db2[v].v[i] = add2(b0.v[i], db2[v].v[i]);
            }
            if (!last_of_team) {
                store_cols<VEC>(p + 2 * (size_t)a.hidden, col(v), n, dw2[v]);
                store_cols<VEC>(p + 3 * (size_t)a.hidden, col(v), n, db2[v]);
                dw2[v] = db2[v] = all8(0.f);
            }
        }
        gates_before = true;
    };
    if (GATE == 2) take_gate();

    // the eight sums of a row, published to every CTA of the team
    auto publish = [&](uint64_t row, uint32_t slot, const GateRow &gr, const float4 &st, uint32_t at) {
        const float2 x1 = both(st.y), x0 = both(-st.x), y0 = both(-st.z);
        float2 s2[kSums];
#pragma unroll
        for (int k = 0; k < kSums; ++k) s2[k] = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Run w = load_run(row, slot, gr, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // xhat = x1 xc, yhat = y1 yc: the scales of a row come to its sums at the end
                const float2 xc = add2(w.r.v[i], x0), yc = add2(w.y.v[i], y0);
                const float2 av = mul2(w1[v].v[i], w.dh.v[i]);
                const float2 base = fma2(x1, av, w.dr.v[i]);
                float2 c = w2[v].v[i];
                if (GATE == 1) c = mul2(c, a.gate_act == BF16OPT_GATE_SIGMOID ? sigmoid2(w.gate.v[i]) : w.gate.v[i]);
                const float2 cy = mul2(c, yc);
                s2[0] = add2(s2[0], av);
                s2[1] = fma2(av, xc, s2[1]);
                s2[2] = fma2(c, base, s2[2]);
                s2[3] = add2(s2[3], c);
                s2[4] = fma2(c, xc, s2[4]);
                s2[5] = fma2(cy, base, s2[5]);
                s2[6] = add2(s2[6], cy);
                s2[7] = fma2(cy, xc, s2[7]);
            }
        }
        float s[kSums];
#pragma unroll
        for (int k = 0; k < kSums; ++k) s[k] = s2[k].x + s2[k].y;
        const float sum = warp_sum8(s, lane);   // value lane_value(lane & 7)
        float *to = sm_sums + at + (rank * warps + warp) * kSums + lane_value(lane & 7);
        if (ranks > 1) {
            for (uint32_t r = lane >> 3; r < ranks; r += 4) *cluster.map_shared_rank(to, r) = sum;   // eight lanes to each rank
        } else if (lane < 8) {
            *to = sum;
        }
    };
    // The sums of all entries, in their order: a lane adds up quarters (four values) of every sixteenth
    // entry, then the lanes join, handing half of their values over while they have more than one.
    auto totals = [&](uint32_t at, float (&s)[kSums]) {
        const float4 *from = reinterpret_cast<const float4 *>(sm_sums + at);
        float4 q4 = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t i = lane; i < 2 * entries; i += 32) {
            const float4 e = from[i];
            q4.x += e.x, q4.y += e.y, q4.z += e.z, q4.w += e.w;
        }
        const bool hi = lane & 16, mid = lane & 8;
        const float2 keep = hi ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y), give = hi ? make_float2(q4.x, q4.y) : make_float2(q4.z, q4.w);
        const float2 h = make_float2(keep.x + __shfl_xor_sync(0xffffffffu, give.x, 16), keep.y + __shfl_xor_sync(0xffffffffu, give.y, 16));
        float one = (mid ? h.y : h.x) + __shfl_xor_sync(0xffffffffu, mid ? h.x : h.y, 8);
        one += __shfl_xor_sync(0xffffffffu, one, 4);
        one += __shfl_xor_sync(0xffffffffu, one, 2);
#pragma unroll
        for (int k = 0; k < kSums; ++k) s[k] = __shfl_sync(0xffffffffu, one, (k >> 2) | ((k >> 1) & 1) << 4 | (k & 1) << 3);
    };

    float4 st = stats_of(row0), st1 = stats_of(row0 + 1);
    uint32_t slot = 0, slot1 = 1;   // the ring is two rows deep at least
    copy_wait_for(depth - 1);
    publish(row0, 0, gate, st, 0);
    if (ranks > 1) cluster_arrive();
    for (uint64_t row = row0; row < row1; ++row) {
        const uint32_t at1 = sums_next(sums_at);
        if (ranks > 1) cluster_wait();
        else __syncthreads();
        // the next row's sums set out before this row's are used
        GateRow gate1 = gate;
        gate_next(gate1);
        const bool gate_over = GATE == 2 && (gate.left == 1 || row + 1 == row1);
        auto publish_next = [&]() {
            if (row + 1 < row1) {
                copy_wait_for(depth - 2);
                publish(row + 1, slot1, gate1, st1, at1);
            }
            if (ranks > 1) cluster_arrive();
        };
        if (!gate_over) publish_next();
        // after the arrival: the release before it waits for loads on their way (205 against 181 us on
        // 4096 x 14336 with these loads at the row's start)
        const float4 st2 = stats_of(row + 2);

        float s[kSums];
        totals(sums_at, s);
        sums_at = at1;
        // g = base - (m1 + xhat m2);  e = c g;  dy = rs2 (e - n1 - yhat n2); the sums are those of xc and yc
        const float m1 = pre_layer ? s[0] * inv_h * st.y : 0.f, m2 = s[1] * st.y * inv_h * st.y;
        const float n1 = post_layer ? (s[2] - m1 * s[3] - m2 * (s[4] * st.y)) * inv_h : 0.f;
        const float n2 = post ? (s[5] - m1 * s[6] - m2 * (s[7] * st.y)) * st.w * inv_h : 0.f;
        const float2 x1 = both(st.y), x0 = both(-st.x), y1 = both(st.w), y0 = both(-st.z);
        const float2 nm1 = both(-m1), nm2 = both(-m2 * st.y), nn1 = both(-n1 * st.w), nn2 = both(-n2 * st.w * st.w);
        // the gate's rows end, here or for this team; its sum is whole if they all are this team's,
        // else a part: of the team's first gate, or of its last
        const uint64_t gate_first = gate.row * a.rows_per_gate;
        const bool gate_ends = GATE == 1 && q.shared_gate && (gate.left == 1 || row + 1 == row1), gate_whole = gate_first >= row0 && gate.left == 1;
        const uint64_t o = row * a.hidden + c0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Run w = load_run(row, slot, gate, v);
            Cols dx, dy, dgr;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 xc = add2(w.r.v[i], x0), yc = add2(w.y.v[i], y0), xdh = mul2(x1, w.dh.v[i]);
                const float2 base = fma2(w1[v].v[i], xdh, w.dr.v[i]);
                float2 g = add2(fma2(xc, nm2, base), nm1);
                dx.v[i] = mul2(rs, g);
                if (GATE == 1) {
                    float2 act = w.gate.v[i];
                    const float2 du = mul2(g, fma2(mul2(yc, y1), w2[v].v[i], b2[v].v[i]));
                    if (a.gate_act == BF16OPT_GATE_SIGMOID) {
                        act = sigmoid2(act);
                        dgr.v[i] = mul2(du, mul2(act, make_float2(1.f - act.x, 1.f - act.y)));
                    } else {
                        dgr.v[i] = du;
                    }
                    g = mul2(act, g);
                }
                const float2 gy = mul2(y1, g);
                dw2[v].v[i] = fma2(gy, yc, dw2[v].v[i]);
                db2[v].v[i] = add2(db2[v].v[i], g);
                dw1[v].v[i] = fma2(xdh, xc, dw1[v].v[i]);
                db1[v].v[i] = add2(db1[v].v[i], w.dh.v[i]);
                dy.v[i] = fma2(w2[v].v[i], gy, fma2(yc, nn2, nn1));
            }
            store_run<VEC>(reinterpret_cast<TS *>(q.dx) + o, col(v), n, dx, lane);
            store_run<VEC>(reinterpret_cast<TB *>(q.dy) + o, col(v), n, dy, lane);
            if (GATE == 1 && q.dgate) {
                if (q.shared_gate) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) dg[v].v[i] = add2(dg[v].v[i], dgr.v[i]);
                    if (gate_ends) {
                        if (gate_whole) store_cols<VEC>(reinterpret_cast<TB *>(q.dgate) + gate.row * a.hidden + c0, col(v), n, dg[v]);
                        else store_cols<VEC>(q.gate_part + (size_t)(2 * team + (gate_first > row0 ? 1 : 0)) * a.hidden + c0, col(v), n, dg[v]);
                        dg[v] = all8(0.f);
                    }
                } else {
                    store_run<VEC>(reinterpret_cast<TB *>(q.dgate) + o, col(v), n, dgr, lane);
                }
            }
        }
        if (gate_over) {
            end_gate(gate.row * a.rows_per_gate >= row0 && gate.left == 1, row + 1 == row1);
            gate = gate1;
            if (row + 1 < row1) take_gate();
            publish_next();
        }
        fill();
        slot = slot1;
        slot1 = slot1 + 1 == depth ? 0 : slot1 + 1;
        st = st1, st1 = st2;
        gate = gate1;
    }
    if (ranks > 1) cluster_wait();   // for the last arrival: nobody leaves while others may write here
    const float2 bs = both(a.branch_scale);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float *p = q.part + (size_t)team * 4 * a.hidden + c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) dw2[v].v[i] = mul2(bs, dw2[v].v[i]), db2[v].v[i] = mul2(bs, db2[v].v[i]);
        if (q.want & 1) store_cols<VEC>(p, col(v), n, dw1[v]);
        if (q.want & 2) store_cols<VEC>(p + a.hidden, col(v), n, db1[v]);
        if (q.want & 4) store_cols<VEC>(p + 2 * (size_t)a.hidden, col(v), n, dw2[v]);
        if (q.want & 8) store_cols<VEC>(p + 3 * (size_t)a.hidden, col(v), n, db2[v]);
    }
    pdl_leave();
}

// The partial sums joined, in the teams' order: 32 columns by kRuns runs of teams.
// blockIdx.y < 4: that weight's gradient; else gate row blockIdx.y - 4, if its
// rows straddle teams.
struct JoinArgs {
    const float *part, *gate_part;
    void *out[4];
    int weight_type, gate_type;
    void *dgate;
    uint64_t rows, gate_rows, rows_per_gate;
    uint32_t teams, hidden;
};
constexpr int kRuns = 16;
template <int W>   // columns of a lane: 4 where the partial sums' rows are whole 16-byte vectors, else 1
__global__ void __launch_bounds__(32 * kRuns) k_norm_join(const JoinArgs j) {
    __shared__ float sm[kRuns][32 * W];
    pdl_enter();
    const uint32_t lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const uint32_t c = (blockIdx.x * 32 + lane) * W;
    for (uint64_t b = blockIdx.y; b < 4 + (j.dgate ? j.gate_rows : 0); b += gridDim.y) {
        const float *p;          // part i is p + i * stride (+ skip for i = 0)
        size_t stride, skip = 0;
        uint32_t count;
        uint64_t at;
        void *out;
        if (b < 4) {
            out = b == 0 ? j.out[0] : b == 1 ? j.out[1] : b == 2 ? j.out[2] : j.out[3];
            p = j.part + b * j.hidden, stride = 4 * (size_t)j.hidden, count = j.teams;
            at = 0;
        } else {
            const uint64_t g = b - 4, first = g * j.rows_per_gate, last = first + j.rows_per_gate - 1;
            const uint32_t p0 = team_of(j.rows, j.teams, first), p1 = team_of(j.rows, j.teams, last);
            out = p0 == p1 ? nullptr : j.dgate;   // within one team: already written
            at = g * j.hidden;
            p = j.gate_part + (size_t)(2 * p0) * j.hidden, stride = 2 * (size_t)j.hidden, count = p1 - p0 + 1;
            skip = first > team_row(j.rows, j.teams, p0) ? j.hidden : 0;   // the first team's last gate, not its first
        }
        if (!out) continue;
        float s[W] = {};
        const uint32_t i0 = count * run / kRuns, i1 = count * (run + 1) / kRuns;
        if (c < j.hidden)
#pragma unroll 8
            for (uint32_t i = i0; i < i1; ++i) {
                const float *from = p + i * stride + (i ? 0 : skip) + c;
                if constexpr (W == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(from);
                    s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
                } else {
                    s[0] += *from;
                }
            }
#pragma unroll
        for (int k = 0; k < W; ++k) sm[run][lane * W + k] = s[k];
        __syncthreads();
        if (threadIdx.x < 32 * W) {   // one thread a column
            const uint32_t column = blockIdx.x * 32 * W + threadIdx.x;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kRuns; ++i) sum += sm[i][threadIdx.x];
            if (column < j.hidden) store_typed(out, b < 4 ? j.weight_type : j.gate_type, at + column, sum);
        }
        __syncthreads();
    }
    pdl_leave();
}

// ---------------------------------------------------------------------- host

int check(const bf16opt_norm_gate_t *d) {
    auto bad = [](const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("norm_gate: ") + m); };
    if (!d) return bad("the descriptor is NULL");
    if (!type_ok(d->branch_type) || !type_ok(d->stream_type) || !type_ok(d->weight_type)) return bad("unknown element type");
    if (d->branch_type == BF16OPT_TYPE_F32 && d->stream_type != BF16OPT_TYPE_F32) return bad("an FP32 branch needs an FP32 stream");
    if (d->hidden < 1 || d->hidden > BF16OPT_NORM_MAX_HIDDEN) return bad("hidden must lie in [1, BF16OPT_NORM_MAX_HIDDEN]");
    if (d->rows >= (1ull << 40)) return bad("too many rows");
    if (d->pre < 0 || d->pre > BF16OPT_NORM_LAYER || d->post < 0 || d->post > BF16OPT_NORM_LAYER) return bad("unknown norm");
    if (d->gate_act != BF16OPT_GATE_IDENTITY && d->gate_act != BF16OPT_GATE_SIGMOID) return bad("unknown gate_act");
    if (d->reserved != 0) return bad("reserved must be 0");
    if (!d->gate != (d->gate_rows == 0)) return bad("gate and gate_rows go together");
    if (d->gate_rows && d->rows % d->gate_rows != 0) return bad("gate_rows must divide rows");
    if (d->gate_rows > d->rows && d->rows) return bad("gate_rows must divide rows");
    if (d->pre == BF16OPT_NORM_NONE && (d->pre_weight || d->pre_bias)) return bad("a weight without its norm (pre)");
    if (d->post == BF16OPT_NORM_NONE && (d->post_weight || d->post_bias)) return bad("a weight without its norm (post)");
    if (!std::isfinite(d->residual_scale) || !std::isfinite(d->branch_scale)) return bad("the scales must be finite");
    if (!std::isfinite(d->eps) || !(d->eps > 0.f)) return bad("eps must be finite and > 0");
    const uint64_t tb = type_bytes(d->branch_type), tw = type_bytes(d->weight_type);
    if (misaligned(d->gate, tb)) return fail(BF16OPT_ERR_ALIGNMENT, "norm_gate: gate is not aligned to its element");
    for (const void *w : {d->pre_weight, d->pre_bias, d->post_weight, d->post_bias})
        if (misaligned(w, tw)) return fail(BF16OPT_ERR_ALIGNMENT, "norm_gate: a weight is not aligned to its element");
    return BF16OPT_OK;
}

struct Part {
    const void *p;
    uint64_t n;
    const void *may = nullptr;   // the input that this output may be
};
int check_overlap(std::initializer_list<Part> outs, std::initializer_list<Part> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Part &x : ins)
            if (overlap(o->p, o->n, x.p, x.n) && !(o->p == x.p && o->may == x.p))
                return fail(BF16OPT_ERR_INVALID_ARG, "norm_gate: an output overlaps an input");
        for (auto e = outs.begin(); e != o; ++e)
            if (overlap(o->p, o->n, e->p, e->n)) return fail(BF16OPT_ERR_INVALID_ARG, "norm_gate: two outputs overlap");
    }
    return BF16OPT_OK;
}

Args args_of(const bf16opt_norm_gate_t *d) {
    Args a;
    a.rows = d->rows, a.hidden = d->hidden, a.weight_type = d->weight_type;
    a.pre = {d->pre, d->pre_weight, d->pre_bias}, a.post = {d->post, d->post_weight, d->post_bias};
    a.gate_act = d->gate_act, a.gate_rows = d->gate_rows, a.rows_per_gate = d->gate_rows ? d->rows / d->gate_rows : 1;
    a.gate = d->gate;
    a.residual_scale = d->residual_scale, a.branch_scale = d->branch_scale, a.eps = d->eps;
    return a;
}

// Whether rows can be moved as 16-byte vectors of eight columns.
bool vectors(const bf16opt_norm_gate_t *d, std::initializer_list<const void *> more) {
    if (d->hidden % 8) return false;
    for (const void *p : {d->gate, d->pre_weight, d->pre_bias, d->post_weight, d->post_bias})
        if (misaligned(p, 16)) return false;
    for (const void *p : more)
        if (misaligned(p, 16)) return false;
    return true;
}

constexpr size_t kSmemBytes = 226 * 1024;   // of a multiprocessor; each CTA takes 1 KB besides its own
// What each of per_sm CTAs can have for its ring besides `other` bytes (at most what a kernel is allowed).
size_t ring_bytes(unsigned per_sm, size_t other) {
    return std::min<size_t>(kSmemBytes / per_sm - 1024, kMaxDynamic) - other;
}

template <class TB, class TS, bool GATE, int V>
int forward_ring(const Args &a, const void *x, const void *y, void *r, void *h, float *stats, cudaStream_t st) {
    auto k = k_norm_forward_ring<TB, TS, GATE, V>;
    const uint32_t threads = ((a.hidden + 8 * V - 1) / (8 * V) + 31) / 32 * 32;
    const size_t row = (size_t)threads * V * 16 * ((GATE ? 2 : 1) * sizeof(TB) / 2 + sizeof(TS) / 2);
    const unsigned per_sm = std::max(1u, std::min((V == 4 ? 512u : 768u) / threads, 16u));   // by the registers
    const uint32_t depth = (uint32_t)std::max<size_t>(1, std::min<size_t>(4, ring_bytes(per_sm, 256) / row));
    Launch l{1, threads, depth * row, st, 1, true};
    int fit = 0;
    cudaError_t e = clusters_that_fit(l, k, fit);
    if (e != cudaSuccess) return fail_cuda(e, "norm_gate occupancy");
    l.grid = (unsigned)std::min<uint64_t>(a.rows, fit);
    l.cluster = 0;
    e = launch(l, k, a, (const TS *)x, (const TB *)y, (TS *)r, (TB *)h, stats, depth);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "norm_gate kernel launch");
}

template <class TB, class TS, bool VEC>
int forward_v(const Args &a, const void *x, const void *y, void *r, void *h, float *stats, cudaStream_t st) {
    const uint32_t vecs = (a.hidden + 7) / 8;
    auto go = [&](auto kernel, unsigned block, bool warp) {
        // a row to each warp or CTA; 2^30 CTAs to a launch (rows walked in a loop instead took 20 to 45 registers more
        // and 17 to 46 % longer)
        constexpr uint64_t kBlocks = 1u << 30;
        for (uint64_t row0 = 0; row0 < a.rows; row0 += kBlocks * (warp ? 4 : 1)) {
            const uint64_t blocks = warp ? (a.rows - row0 + 3) / 4 : a.rows - row0;
            Launch l{(unsigned)std::min(blocks, kBlocks), block, 0, st, 0, true};
            const cudaError_t e = launch(l, kernel, a, (const TS *)x, (const TB *)y, (TS *)r, (TB *)h, stats, row0);
            if (e != cudaSuccess) return fail_cuda(e, "norm_gate kernel launch");
        }
        return BF16OPT_OK;
    };
    if (vecs <= 32) return go(k_norm_forward<TB, TS, VEC, true, 1>, 128, true);
    if (vecs <= 64) return go(k_norm_forward<TB, TS, VEC, true, 2>, 128, true);
    if constexpr (VEC) {
        auto ring = [&](auto v) {
            constexpr int V = decltype(v)::value;
            return a.gate ? forward_ring<TB, TS, true, V>(a, x, y, r, h, stats, st) : forward_ring<TB, TS, false, V>(a, x, y, r, h, stats, st);
        };
        return vecs <= 768 ? ring(std::integral_constant<int, 2>()) : ring(std::integral_constant<int, 4>());
    } else {
        auto block = [&](uint32_t nv) { return (unsigned)(((vecs + nv - 1) / nv + 31) / 32 * 32); };
        if (vecs <= 512) return go(k_norm_forward<TB, TS, VEC, false, 1>, block(1), false);
        if (vecs <= 1024) return go(k_norm_forward<TB, TS, VEC, false, 2>, block(2), false);
        return go(k_norm_forward<TB, TS, VEC, false, 4>, block(4), false);
    }
}

// The backward pass's shape, from the sizes and the device alone.
struct Shape {
    unsigned cluster, threads;
    uint32_t depth;          // rows in the ring
    size_t smem;
    uint32_t teams;
    uint64_t part_floats, gate_floats;
};

template <class F>
int by_types(const bf16opt_norm_gate_t *d, F &&f) {
    using B = __nv_bfloat16;
    if (d->branch_type == BF16OPT_TYPE_F32) return f((float *)nullptr, (float *)nullptr);
    if (d->stream_type == BF16OPT_TYPE_F32) return f((B *)nullptr, (float *)nullptr);
    return f((B *)nullptr, (B *)nullptr);
}

// Runs of eight columns a thread has: two where whole vectors pass through the ring, and
// no gate comes with every row (its sums would not fit the registers).
template <bool VEC, int GATE>
constexpr int runs_of() { return VEC && GATE != 1 ? 2 : 1; }

template <class TB, class TS, bool VEC, int GATE>
int shape_v(const bf16opt_norm_gate_t *d, Shape &s) {
    constexpr int V = runs_of<VEC, GATE>();
    // CTAs that share the columns: so many that a CTA's fit its threads, and two rows of them its ring; and
    // more where the SM then holds half as many threads again (8192 x 4097: two CTAs of 288 threads, one
    // per SM, 340 us; four of 160, three per SM, 281 us).
    size_t row = 0, sums = 0;
    auto per_sm_of = [](uint32_t threads) { return std::max(1u, std::min(512u / threads, 16u)); };   // 128 registers a thread
    auto threads_of = [&](uint32_t cluster) {
        const uint32_t cols = (d->hidden + cluster - 1) / cluster;
        return ((cols + 8 * V - 1) / (8 * V) + 31) / 32 * 32;
    };
    for (s.cluster = 1;; s.cluster *= 2) {
        s.threads = threads_of(s.cluster);
        row = (size_t)s.threads * V * ring_units<TB, TS, VEC, GATE>() * 16;
        sums = 3 * s.cluster * s.threads / 32 * kSums * sizeof(float);
        if (s.threads > (uint32_t)kBackThreads || 2 * row + sums > kMaxDynamic) continue;
        const uint32_t half = threads_of(2 * s.cluster);
        if (s.cluster < 8 && 2 * half * per_sm_of(half) >= 3 * s.threads * per_sm_of(s.threads)) continue;
        break;
    }
    const unsigned per_sm = per_sm_of(s.threads);
    s.depth = (uint32_t)std::max<size_t>(2, std::min<size_t>(8, ring_bytes(per_sm, sums) / row));
    s.smem = s.depth * row + sums;
    int fit = 0;
    const cudaError_t e = clusters_that_fit(Launch{s.cluster, s.threads, s.smem, nullptr, s.cluster, true},
                                            k_norm_backward<TB, TS, VEC, GATE, V>, fit);
    if (e != cudaSuccess) return fail_cuda(e, "norm_gate occupancy");
    const uint64_t teams = fit;
    s.teams = (uint32_t)std::min<uint64_t>(teams, std::max<uint64_t>(1, d->rows));
    s.part_floats = (uint64_t)s.teams * 4 * d->hidden;
    s.gate_floats = d->gate_rows && d->gate_rows != d->rows ? (uint64_t)s.teams * 2 * d->hidden : 0;
    return BF16OPT_OK;
}
// How the backward pass has the gate (k_norm_backward's GATE).
int gate_kind(const bf16opt_norm_gate_t *d) {
    return !d->gate ? 0 : d->rows / d->gate_rows < kGateRows ? 1 : 2;
}
template <class TB, class TS>
int shape_t(const bf16opt_norm_gate_t *d, bool vec, Shape &s) {
    switch (gate_kind(d)) {
    case 0: return vec ? shape_v<TB, TS, true, 0>(d, s) : shape_v<TB, TS, false, 0>(d, s);
    case 1: return vec ? shape_v<TB, TS, true, 1>(d, s) : shape_v<TB, TS, false, 1>(d, s);
    default: return vec ? shape_v<TB, TS, true, 2>(d, s) : shape_v<TB, TS, false, 2>(d, s);
    }
}

template <class TB, class TS, bool VEC, int GATE>
int backward_v(const Args &a, const BackArgs &q, const Shape &s, cudaStream_t st) {
    auto k = k_norm_backward<TB, TS, VEC, GATE, runs_of<VEC, GATE>()>;
    Launch l{s.teams * s.cluster, s.threads, s.smem, st, s.cluster, true};
    const cudaError_t e = launch(l, k, a, q, s.depth);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "norm_gate kernel launch");
}

int forward(const bf16opt_norm_gate_t *d, const void *x, const void *y, void *r, void *h, float *stats, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    const bool pre = d->pre != BF16OPT_NORM_NONE;
    if (d->rows && (!x || !y || !r || (pre && !h))) return fail(BF16OPT_ERR_INVALID_ARG, "norm_gate: x, y, r or h is NULL");
    if (!pre && h) return fail(BF16OPT_ERR_INVALID_ARG, "norm_gate: h without a norm (pre)");
    if (d->rows == 0) return BF16OPT_OK;
    const uint64_t tb = type_bytes(d->branch_type), ts = type_bytes(d->stream_type), tw = type_bytes(d->weight_type);
    if (misaligned(x, ts) || misaligned(r, ts) || misaligned(y, tb) || misaligned(h, tb) || misaligned(stats, 4))
        return fail(BF16OPT_ERR_ALIGNMENT, "norm_gate: a pointer is not aligned to its element");
    const uint64_t n = d->rows * d->hidden, hw = d->hidden * tw;
    rc = check_overlap({{r, n * ts, x}, {h, n * tb, y}, {stats, d->rows * 16}},
                       {{x, n * ts}, {y, n * tb}, {d->gate, d->gate_rows * d->hidden * tb}, {d->pre_weight, hw},
                        {d->pre_bias, hw}, {d->post_weight, hw}, {d->post_bias, hw}});
    if (rc != BF16OPT_OK) return rc;
    if (sm_count() < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "norm_gate: no CUDA device");
    const Args a = args_of(d);
    const cudaStream_t st = (cudaStream_t)stream;
    const bool vec = vectors(d, {x, y, r, h});
    return by_types(d, [&](auto bp, auto tp) {
        using TB = std::remove_pointer_t<decltype(bp)>;
        using TS = std::remove_pointer_t<decltype(tp)>;
        return vec ? forward_v<TB, TS, true>(a, x, y, r, h, stats, st) : forward_v<TB, TS, false>(a, x, y, r, h, stats, st);
    });
}

int workspace(const bf16opt_norm_gate_t *d, uint64_t *bytes) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    const int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    if (!bytes) return fail(BF16OPT_ERR_INVALID_ARG, "norm_gate: bytes is NULL");
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "norm_gate: no CUDA device");
    // the larger of what aligned and other rows take: the pointers are not known yet
    Shape s[2];
    for (int vec = 0; vec < 2; ++vec) {
        const int r = by_types(d, [&](auto b, auto t) {
            return shape_t<std::remove_pointer_t<decltype(b)>, std::remove_pointer_t<decltype(t)>>(d, vec, s[vec]);
        });
        if (r != BF16OPT_OK) return r;
    }
    *bytes = std::max(s[0].part_floats + s[0].gate_floats, s[1].part_floats + s[1].gate_floats) * 4;
    return BF16OPT_OK;
}

int backward(const bf16opt_norm_gate_t *d, const void *dr, const void *dh, const void *r, const void *y, const float *stats,
             void *dx, void *dy, void *dgate, void *dpre_weight, void *dpre_bias, void *dpost_weight, void *dpost_bias,
             void *ws, uint64_t ws_bytes, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    auto bad = [](const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("norm_gate: ") + m); };
    const bool pre = d->pre != BF16OPT_NORM_NONE, post = d->post != BF16OPT_NORM_NONE;
    if ((dpre_weight && !d->pre_weight) || (dpre_bias && !d->pre_bias) || (dpost_weight && !d->post_weight) ||
        (dpost_bias && !d->post_bias) || (dgate && !d->gate))
        return bad("a gradient of a weight that is not there");
    if (!pre && dh) return bad("dh without a norm (pre)");
    if (d->rows && (!y || !dx || !dy || (dh && !r) || ((pre || post) && !stats))) return bad("r, y, stats, dx or dy is NULL");
    const uint64_t tb = type_bytes(d->branch_type), ts = type_bytes(d->stream_type), tw = type_bytes(d->weight_type);
    void *const outs[4] = {dpre_weight, dpre_bias, dpost_weight, dpost_bias};
    uint32_t want = 0;
    for (int i = 0; i < 4; ++i) {
        void *const w = outs[i];
        want |= w ? 1u << i : 0u;
        if (misaligned(w, tw)) return fail(BF16OPT_ERR_ALIGNMENT, "norm_gate: a pointer is not aligned to its element");
    }
    if (misaligned(dr, ts) || misaligned(r, ts) || misaligned(dx, ts) || misaligned(dh, tb) || misaligned(y, tb) ||
        misaligned(dy, tb) || misaligned(dgate, tb) || misaligned(stats, 4) || misaligned(ws, 16))
        return fail(BF16OPT_ERR_ALIGNMENT, "norm_gate: a pointer is not aligned to its element (workspace: 16 bytes)");
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "norm_gate: no CUDA device");
    const cudaStream_t st = (cudaStream_t)stream;
    if (d->rows == 0) {
        cudaError_t e = cudaSuccess;
        for (void *w : outs)
            if (w && e == cudaSuccess) e = cudaMemsetAsync(w, 0, d->hidden * tw, st);
        if (dgate && e == cudaSuccess) e = cudaMemsetAsync(dgate, 0, d->gate_rows * d->hidden * tb, st);
        return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "norm_gate clearing the weights' gradients");
    }
    const bool vec = vectors(d, {dr, dh, r, y, dx, dy, dgate});
    Shape s;
    rc = by_types(d, [&](auto b, auto t) {
        return shape_t<std::remove_pointer_t<decltype(b)>, std::remove_pointer_t<decltype(t)>>(d, vec, s);
    });
    if (rc != BF16OPT_OK) return rc;
    const uint64_t ws_need = (s.part_floats + s.gate_floats) * 4;
    if (!ws || ws_bytes < ws_need) return bad("the workspace is too small");
    const uint64_t n = d->rows * d->hidden, hw = d->hidden * tw, gb = d->gate_rows * d->hidden * tb;
    rc = check_overlap({{dx, n * ts, dr}, {dy, n * tb, dh}, {dgate, gb}, {dpre_weight, hw}, {dpre_bias, hw},
                        {dpost_weight, hw}, {dpost_bias, hw}, {ws, ws_need}},
                       {{dr, n * ts}, {dh, n * tb}, {r, n * ts}, {y, n * tb}, {stats, d->rows * 16}, {d->gate, gb},
                        {d->pre_weight, hw}, {d->pre_bias, hw}, {d->post_weight, hw}, {d->post_bias, hw}});
    if (rc != BF16OPT_OK) return rc;
    Args a = args_of(d);
    BackArgs q;
    q.dr = dr, q.dh = dh, q.r = r, q.y = y, q.stats = stats, q.dx = dx, q.dy = dy, q.dgate = dgate;
    q.part = (float *)ws, q.gate_part = (float *)ws + s.part_floats;
    q.teams = s.teams, q.want = want;
    q.shared_gate = dgate && d->gate_rows != d->rows;
    rc = by_types(d, [&](auto bp, auto tp) {
        using TB = std::remove_pointer_t<decltype(bp)>;
        using TS = std::remove_pointer_t<decltype(tp)>;
        switch (gate_kind(d)) {
        case 0: return vec ? backward_v<TB, TS, true, 0>(a, q, s, st) : backward_v<TB, TS, false, 0>(a, q, s, st);
        case 1: return vec ? backward_v<TB, TS, true, 1>(a, q, s, st) : backward_v<TB, TS, false, 1>(a, q, s, st);
        default: return vec ? backward_v<TB, TS, true, 2>(a, q, s, st) : backward_v<TB, TS, false, 2>(a, q, s, st);
        }
    });
    if (rc != BF16OPT_OK || (!want && !q.shared_gate)) return rc;
    JoinArgs j;
    j.part = q.part, j.gate_part = q.gate_part;
    for (int i = 0; i < 4; ++i) j.out[i] = outs[i];
    j.weight_type = d->weight_type, j.gate_type = d->branch_type;
    j.dgate = q.shared_gate ? dgate : nullptr;
    j.rows = a.rows, j.gate_rows = a.gate_rows, j.rows_per_gate = a.rows_per_gate;
    j.teams = s.teams, j.hidden = a.hidden;
    // four columns a lane where that leaves a block for every SM (14336 columns: 18 us against 6 us; 2048: 6 against 10)
    const uint32_t width = a.hidden % 4 == 0 && a.hidden >= 32u * (unsigned)sms ? 4 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.hidden + 32 * width - 1) / (32 * width), (unsigned)std::min<uint64_t>(4 + (j.dgate ? a.gate_rows : 0), 4096));
    cfg.blockDim = dim3(32 * kRuns), cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    const cudaError_t e = width == 4 ? cudaLaunchKernelEx(&cfg, k_norm_join<4>, j) : cudaLaunchKernelEx(&cfg, k_norm_join<1>, j);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "norm_gate kernel launch");
}

}  // namespace
}  // namespace bf16ops

extern "C" int bf16opt_norm_gate_forward(const bf16opt_norm_gate_t *d, const void *x, const void *y, void *r, void *h,
                                         float *stats, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::forward(d, x, y, r, h, stats, stream); });
}

extern "C" int bf16opt_norm_gate_workspace(const bf16opt_norm_gate_t *d, uint64_t *bytes) {
    return bf16ops::guarded([&] { return bf16ops::workspace(d, bytes); });
}

extern "C" int bf16opt_norm_gate_backward(const bf16opt_norm_gate_t *d, const void *dr, const void *dh, const void *r,
                                          const void *y, const float *stats, void *dx, void *dy, void *dgate,
                                          void *dpre_weight, void *dpre_bias, void *dpost_weight, void *dpost_bias,
                                          void *workspace, uint64_t workspace_bytes, void *stream) {
    return bf16ops::guarded([&] {
        return bf16ops::backward(d, dr, dh, r, y, stats, dx, dy, dgate, dpre_weight, dpre_bias, dpost_weight, dpost_bias,
                                 workspace, workspace_bytes, stream);
    });
}
