// glu.cu -- activations kept in 8 bits (bf16opt_pack, bf16opt_unpack) and a feed-forward block's
// activation that keeps its inputs so (bf16opt_glu_*), of include/bf16opt.h.
//
// Everything here is element by element but for a run's largest magnitude, and is bound by its bytes: per
// element of bf16, forward 2 (read) + 1 + 1/32 (kept) for gate and for up and 2 for h;
// backward 2 (dh) + the same kept ones, and 2 for each gradient.
//
// A scale is a power of two, so dividing by it is exact and a code depends on nothing but the
// element and its run's largest: no rounding but the one to e4m3 (half a step of three bits, 2^-4
// relative at most; of what is below 2^-6 scales, 2^-10 scales).
//
// Measured on one GB300 (a copy runs at 6.69 TB/s): 2048 x 57344 bf16, silu, gated, forward 143 us and backward 160 us, 6.2
// TB/s together; 8192 x 8192 gelu backward 95 us, 5.7 TB/s; 4096 x 8192 FP32 gelu both ways 152 us, 6.2 TB/s; 8192 x 14336 bf16
// packed and unpacked 116 us, 6.1 TB/s.  Loads wait for memory (9 to 11 cycles an issue) at 52 to 60 % of the issue slots.  Rows
// between 16-byte boundaries take twice the instructions: 2213 x 18799 both ways 225 us, 3 TB/s.  With a gate, the backward kernels of bf16 and
// the forward ones of rows between boundaries spill (32 to 104 bytes).
#include "ops_common.cuh"

namespace bf16ops {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kRun = BF16OPT_PACK_RUN;

struct Rows {
    const void *p;
    uint64_t stride;   // elements
};

struct Args {
    Rows x[2];         // forward: gate, up; backward: dh
    void *out[3];      // forward: h; backward: dgate, dup, h
    uint64_t out_stride[3];
    uint8_t *codes, *scales;
    uint64_t rows;
    uint32_t columns, runs;   // of a row
    // A CTA has `width` threads side by side along a row (of which there are `blocks` such pieces), `deep` rows at a time.
    uint32_t width, blocks, deep;
};

// ------------------------------------------------------------------ a run's scale

// The scale's byte for a run whose largest finite magnitude has the bits `m`: its exponent less 8, one
// more where the fraction is above 1.75 (448 = 1.75 * 2^8), and no less than 0.  It grows with m, so a run's is the
// largest of its parts'.
__device__ __forceinline__ uint32_t scale_byte(float m) {
    const uint32_t e = (__float_as_uint(m) + 0x1fffffu) >> 23;
    return e > 8 ? e - 8 : 0u;
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 1u << 22); }   // 2^(byte - 127)
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// What would be rounded to 2^128 is kept as the number below it, 1.875 2^127; an infinity as NaN.  Only a run
// with the largest byte there is, which an infinity gives too, may have either.
constexpr uint32_t kLargestByte = 247;
__device__ __forceinline__ float holdable(float x) {
    return fabsf(x) < 0x1.fp127f ? x : fabsf(x) < INFINITY ? copysignf(0x1.ep127f, x) : NAN;
}

// Two floats to e4m3, the first in the low byte (NaN stays NaN), and back, exact in fp16.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_codes(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float2 f;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

// ------------------------------------------------------------------ the activation

__device__ __forceinline__ float reciprocal(float x) {   // 0 above 2^126
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// act(g) = g s, s = sigmoid(y), y = g (silu) or g (a + b g^2), a = 2 sqrt(2 / pi), b = 0.044715 a (gelu: (1 + tanh(y / 2)) / 2 =
// sigmoid(y)); act'(g) = s + g y' s (1 - s).  The exponential is off by 2^-22 and by its argument's rounding, |y| 2^-23 or so, the
// reciprocal by 2^-23, both the special-function unit's for FP32 too (whole outputs are 1.9e-7 off, 8e-8 by torch's functions in
// FP32); 1 - s as a difference is off by 2^-24, which is |g y'| 2^-24 of act' (|y| 2^-24 for silu, up to three times that for
// gelu).  From |g| = 64 on gelu's sigmoid is 0 or 1, and g^2 stops growing.  (NaN goes through g.)
// 1 + exp(-y) is taken 2^-32 times, so that its reciprocal is a normal number as long as the exponential is finite: a sigmoid
// down to 2^-128 counts, which times g is a normal number (silu(-88) = -5e-37).
template <int ACT>
__device__ __forceinline__ float2 activate(float2 g, float2 &slope) {
    constexpr float kA = 1.59576912160573071f, kB = 0.044715f * kA, kSmall = 0x1p-32f;
    float2 y = g, dy = both(1.f);
    if (ACT == BF16OPT_GLU_GELU) {
        float2 q = mul2(g, g);
        q = make_float2(fminf(q.x, 4096.f), fminf(q.y, 4096.f));
        y = mul2(g, fma2(q, both(kB), both(kA)));
        dy = fma2(q, both(3.f * kB), both(kA));
    }
    const float2 x = mul2(y, both(-kLog2e)), t = fma2(make_float2(ex2(x.x), ex2(x.y)), both(kSmall), both(kSmall));
    const float2 s = mul2(make_float2(reciprocal(t.x), reciprocal(t.y)), both(kSmall));
    float2 w = mul2(s, fma2(s, both(-1.f), both(1.f)));
    if (ACT == BF16OPT_GLU_GELU) w = mul2(w, dy);
    slope = fma2(g, w, s);
    return mul2(g, s);
}

// ------------------------------------------------------------------ eight columns of a thread

// Eight neighbours from `first`, four lanes to a run.  ALIGNED: rows begin on 16 bytes.  Otherwise the warp has 256 neighbours of
// one row: each lane reads the aligned vectors that hold its columns, and writes the aligned 16 bytes (32 of FP32) that
// hold its first column, with what the lane before it has of them; nothing but a warp's two ends is written element by element.
template <class T, bool ALIGNED>
struct Eight {
    static constexpr int W = sizeof(T) / 2, N = 8 / W, K = 4 * W;   // vectors; elements of a vector; words
    union {
        uint4 v[W];
        uint32_t w[K];
        T e[8];
    };
    __device__ __forceinline__ Eight() {}

    // Eight elements of x (2 K words) from element t on, 0 <= t < 8.
    __device__ __forceinline__ static void window(uint32_t (&x)[2 * K], uint32_t t, Eight &to) {
        if constexpr (sizeof(T) == 4) {
            if (t & 4)
#pragma unroll
                for (int i = 0; i < 11; ++i) x[i] = x[i + 4];
            if (t & 2)
#pragma unroll
                for (int i = 0; i < 9; ++i) x[i] = x[i + 2];
#pragma unroll
            for (int i = 0; i < 8; ++i) to.w[i] = t & 1 ? x[i + 1] : x[i];
        } else {
            if (t & 4)
#pragma unroll
                for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
            if (t & 2)
#pragma unroll
                for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) to.w[i] = t & 1 ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
        }
    }
    // Elements between the 16-byte boundary before it and p.
    __device__ __forceinline__ static uint32_t beyond(const T *p) { return (uint32_t)((uintptr_t)p & 15u) / (uint32_t)sizeof(T); }

    __device__ __forceinline__ void store(T *row, uint32_t first, uint32_t columns) const {
        const uint32_t s = ALIGNED ? 0 : beyond(row);
        if (ALIGNED || s == 0) {
            if (first + 8 <= columns) {
#pragma unroll
                for (int i = 0; i < W; ++i) __stcs(reinterpret_cast<uint4 *>(row + first) + i, v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (first + i < columns) row[first + i] = e[i];
            }
            return;
        }
        const uint32_t lane = threadIdx.x & 31;
        uint32_t x[2 * K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            x[i] = i < K - 4 ? 0 : __shfl_up_sync(0xffffffffu, w[i], 1);   // (less than a vector of them)
            x[K + i] = w[i];
        }
        Eight block;   // columns [first - s, first - s + 8): its own first 8 - s, behind the last s of the lane before
        window(x, 8 - s, block);
        const bool mine = lane > 0 && first - s + 8 <= columns, next = lane < 31 && first - s + 16 <= columns;
        if (mine) {
#pragma unroll
            for (int i = 0; i < W; ++i) __stcs(reinterpret_cast<uint4 *>(row + (first - s)) + i, block.v[i]);
        }
        // its own elements that neither its vectors nor the next lane's have
        const uint32_t split = (1u << (8 - s)) - 1, valid = first + 8 <= columns ? 0xffu : first < columns ? (1u << (columns - first)) - 1 : 0u;
        const uint32_t left = ((mine ? 0 : split) | (next ? 0 : 0xffu & ~split)) & valid;
        if (left) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (left >> i & 1) row[first + i] = e[i];
        }
    }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
    __device__ __forceinline__ void pack(const float2 (&f)[4]) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16(f[i].x, f[i].y);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[2 * i] = __float_as_uint(f[i].x), w[2 * i + 1] = __float_as_uint(f[i].y);
        }
    }

    // Up to n (8 or a vector's) elements of a row from column `at` on, an aligned address, as vectors where they all are the row's; 0 else.
    __device__ __forceinline__ void piece(const T *row, int32_t at, int n, uint32_t columns) {
        if (at >= 0 && at + n <= (int32_t)columns) {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (i * N < n) v[i] = __ldcs(reinterpret_cast<const uint4 *>(row + at) + i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < n && at + i >= 0 && at + i < (int32_t)columns) e[i] = row[at + i];
                else from_f32(e[i], 0.f);
            }
        }
    }
};

// Columns [first, first + 8) of a row on their way, 0 behind its end.
template <class T, bool ALIGNED>
struct Coming {
    using E = Eight<T, ALIGNED>;
    E block;
    uint32_t s;                   // elements beyond a boundary
    Eight<T, ALIGNED> behind;     // the next vector (s of its elements are wanted, less than it has), which the next lane has too
    __device__ __forceinline__ void ask(const T *row, uint32_t first, uint32_t columns) {
        if (ALIGNED) {
            block.piece(row, (int32_t)first, 8, columns);
        } else {
            s = E::beyond(row);
            block.piece(row, (int32_t)(first - s), 8, columns);
            if (s) behind.piece(row, (int32_t)(first - s + 8), E::N, columns);
        }
    }
    __device__ __forceinline__ E take() const {
        if (ALIGNED || s == 0) return block;
        constexpr int K = E::K;
        uint32_t x[2 * K];
#pragma unroll
        for (int i = 0; i < K; ++i) x[i] = block.w[i], x[K + i] = i < 4 ? behind.w[i] : 0;
        E e;
        E::window(x, s, e);
        return e;
    }
};

// A thread's columns, and the rows that it walks down: the CTA's first one, then every `step`-th.
struct Place {
    uint32_t first, run;   // first column; its run in the row
    bool there;            // the thread has columns within the row's runs
    uint32_t row, step;
};
__device__ __forceinline__ Place place_of(const Args &a) {
    const uint32_t group = blockIdx.x / a.blocks, block = blockIdx.x - group * a.blocks;
    const uint32_t slot = threadIdx.x / a.width, i = block * a.width + (threadIdx.x - slot * a.width);
    Place p;
    p.first = i * 8;
    p.run = p.first / kRun;
    p.there = p.first < a.runs * kRun && slot < a.deep;
    p.row = group * a.deep + slot;
    p.step = gridDim.x / a.blocks * a.deep;
    return p;
}

// Keeps the thread's columns of one row.  Every lane of the warp takes part; `there`: it has any.
template <int PARTS>
__device__ __forceinline__ void keep(const Args &a, const float2 (&f)[PARTS][4], uint8_t *codes, uint8_t *scales, const Place &p, bool there) {
    uint32_t bytes = 0;   // of gate and of up, 16 bits each
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(f[k][i].x), fabsf(f[k][i].y)));   // NaN passed over
        bytes |= scale_byte(m) << (16 * k);
    }
    bytes = __vmaxu2(bytes, __shfl_xor_sync(0xffffffffu, bytes, 1));
    bytes = __vmaxu2(bytes, __shfl_xor_sync(0xffffffffu, bytes, 2));
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        uint32_t byte = bytes >> (16 * k) & 0xffffu;
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f[k][i];
        if (__any_sync(0xffffffffu, byte >= kLargestByte)) {   // the largest finite one again
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m = fmaxf(m, fmaxf(fabsf(x[i].x) < INFINITY ? fabsf(x[i].x) : 0.f, fabsf(x[i].y) < INFINITY ? fabsf(x[i].y) : 0.f));
                x[i] = make_float2(holdable(x[i].x), holdable(x[i].y));
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            byte = scale_byte(fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2)));
        }
        const float2 inv = both(inverse_scale(byte));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], inv);
        uint2 c;
        c.x = to_codes(x[0].x, x[0].y) | to_codes(x[1].x, x[1].y) << 16;
        c.y = to_codes(x[2].x, x[2].y) | to_codes(x[3].x, x[3].y) << 16;
        if (there) {
            __stcs(reinterpret_cast<uint2 *>(codes + k * a.rows * a.runs * kRun), c);
            if ((p.first & (kRun - 1)) == 0) scales[k * a.rows * a.runs] = (uint8_t)byte;
        }
    }
}

// Eight columns of what was kept, on their way.
struct Kept {
    uint2 c;
    uint32_t byte;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scale) {
        c = __ldcs(reinterpret_cast<const uint2 *>(codes));
        byte = *scale;
    }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        const float2 s = both(scale_of(byte));
        f[0] = mul2(from_codes(c.x & 0xffffu), s), f[1] = mul2(from_codes(c.x >> 16), s);
        f[2] = mul2(from_codes(c.y & 0xffffu), s), f[3] = mul2(from_codes(c.y >> 16), s);
    }
};

// ------------------------------------------------------------------ the kernels

// A thread has its columns and walks down the rows with them, `U` rows at a time, the next ones on their way while it
// works on these: addresses only go on by a stride.  U: so many that 32 bytes or so of each thread are on their way.

// PARTS: 1 or 2 of what is kept; ACT < 0: nothing but keeping or reading.
template <class T, bool ALIGNED, int PARTS, int ACT, bool KEEP>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) k_forward(const Args a) {
    constexpr int U = sizeof(T) == 2 && PARTS == 1 && ALIGNED ? 2 : 1;
    using E = Eight<T, ALIGNED>;
    pdl_enter();
    const Place p = place_of(a);
    const T *x[PARTS];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) x[k] = reinterpret_cast<const T *>(a.x[k].p) + p.row * a.x[k].stride;
    T *h = reinterpret_cast<T *>(a.out[0]) + p.row * a.out_stride[0];
    uint8_t *codes = a.codes + (uint64_t)p.row * a.runs * kRun + p.first, *scales = a.scales + (uint64_t)p.row * a.runs + p.run;
    Coming<T, ALIGNED> next[U][PARTS];
    auto ask = [&](uint32_t row) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                if (ALIGNED) next[u][k].ask(x[k], p.there && row + u * p.step < a.rows ? p.first : a.columns, a.columns);
                else if (row + u * p.step < a.rows) next[u][k].ask(x[k], p.first, a.columns);   // (the same in the warp)
                x[k] += p.step * a.x[k].stride;
            }
        }
    };
    ask(p.row);
    // (the same number of turns for the whole CTA: its lanes look at one another's columns)
    for (uint32_t row = p.row, top = p.row - threadIdx.x / a.width; top < a.rows; row += U * p.step, top += U * p.step) {
        float2 f[U][PARTS][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) next[u][k].take().unpack(f[u][k]);
        ask(row + U * p.step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool there = p.there && row + u * p.step < a.rows;
            if (ACT >= 0) {
                float2 v[4], slope;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = activate<ACT>(f[u][0][i], slope);
                    if (PARTS > 1) v[i] = mul2(v[i], f[u][PARTS - 1][i]);
                }
                E e;
                e.pack(v);
                if (ALIGNED ? there : row + u * p.step < a.rows) e.store(h, p.first, a.columns);
                h += p.step * a.out_stride[0];
            }
            if (KEEP) {
                keep<PARTS>(a, f[u], codes, scales, p, there);
                codes += (uint64_t)p.step * a.runs * kRun, scales += (uint64_t)p.step * a.runs;
            }
        }
    }
    pdl_leave();
}

// Two gradients and what is kept leave few registers: of bf16 five CTAs of an SM ask for a row when they have written the last one,
// which beats four that ask before (2048 x 57344: 160 against 165 us); of FP32 three that ask before (4096 x 8192: 79 against
// 91 us).  (A ring of asynchronous copies, two to four rows ahead, took 161 and 98 us.)
template <class T, bool ALIGNED, int PARTS, int ACT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : ALIGNED && ACT >= 0 ? 5 : 4) k_backward(const Args a) {
    constexpr int U = ACT < 0 && ALIGNED ? 4 : 1;
    constexpr bool kBefore = sizeof(T) == 4 || !ALIGNED || ACT < 0;
    using E = Eight<T, ALIGNED>;
    pdl_enter();
    const Place p = place_of(a);
    if (ALIGNED && !p.there) return;   // (otherwise a warp's lanes, of one row, stay together)
    const T *x = reinterpret_cast<const T *>(a.x[0].p) + p.row * a.x[0].stride;
    const uint8_t *codes = a.codes + (uint64_t)p.row * a.runs * kRun + p.first, *scales = a.scales + (uint64_t)p.row * a.runs + p.run;
    Coming<T, ALIGNED> next;
    Kept kept[U][PARTS] = {};
    auto ask = [&](uint32_t row) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row + u * p.step < a.rows) {
                if (ACT >= 0) next.ask(x, p.first, a.columns);
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
                    if (ALIGNED || p.there) kept[u][k].load(codes + k * a.rows * a.runs * kRun, scales + k * a.rows * a.runs);
            }
            if (ACT >= 0) x += p.step * a.x[0].stride;
            codes += (uint64_t)p.step * a.runs * kRun, scales += (uint64_t)p.step * a.runs;
        }
    };
    ask(p.row);
    for (uint32_t row = p.row; row < a.rows; row += U * p.step) {
        float2 f[U][PARTS][4], dh[4];
        if (ACT >= 0) next.take().unpack(dh);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) kept[u][k].unpack(f[u][k]);
        if (kBefore) ask(row + U * p.step);
        auto put = [&](int i, uint32_t r, const float2 (&v)[4]) {
            E e;
            e.pack(v);
            e.store(reinterpret_cast<T *>(a.out[i]) + r * a.out_stride[i], p.first, a.columns);
        };
        if constexpr (ACT < 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (row + u * p.step < a.rows) put(0, row + u * p.step, f[u][0]);
        } else {
            float2 dg[4], du[4], h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 slope;
                h[i] = activate<ACT>(f[0][0][i], slope);
                dg[i] = mul2(dh[i], slope);
                if (PARTS > 1) {
                    dg[i] = mul2(dg[i], f[0][PARTS - 1][i]);
                    du[i] = mul2(dh[i], h[i]);
                    h[i] = mul2(h[i], f[0][PARTS - 1][i]);
                }
            }
            put(0, row, dg);
            if (PARTS > 1) put(1, row, du);
            if (a.out[2]) put(2, row, h);
        }
        if (!kBefore) ask(row + U * p.step);
    }
    pdl_leave();
}

// ---------------------------------------------------------------------- host

int bad(const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("glu: ") + m); }

struct Tensor {   // rows of an activation
    const void *p;
    uint64_t stride;
    bool out;
};

// Everything that both directions ask of their arguments; `skip`: nothing to do.
int check(uint64_t rows, uint32_t columns, int type, uint32_t parts, std::initializer_list<Tensor> tensors, const uint8_t *codes,
          const uint8_t *scales, bool writes_codes, bool &skip) {
    skip = false;
    if (!type_ok(type)) return bad("unknown element type");
    if (columns < 1 || columns > (1u << 30)) return bad("columns must lie in [1, 2^30]");
    const uint64_t e = type_bytes(type);
    uint64_t bytes = 0;
    for (const Tensor &t : tensors) {
        if (t.stride < columns) return bad("a row stride is below columns");
        if (!span_bytes(rows, t.stride, columns, e, bytes)) return bad("the sizes overflow");
    }
    const uint64_t runs = (columns + kRun - 1) / kRun;
    if (rows >= (1ull << 31) || !span_bytes(rows, runs * kRun * parts, runs * kRun * parts, 1, bytes)) return bad("the sizes overflow");
    if (rows == 0) {
        skip = true;
        return BF16OPT_OK;
    }
    for (const Tensor &t : tensors) {
        if (!t.p) return bad("a pointer is NULL");
        if (misaligned(t.p, e)) return fail(BF16OPT_ERR_ALIGNMENT, "glu: a pointer is not aligned to its element");
    }
    if (codes && misaligned(codes, 16)) return fail(BF16OPT_ERR_ALIGNMENT, "glu: codes must be 16-byte aligned");
    const uint64_t nc = parts * rows * runs * kRun, ns = parts * rows * runs;
    if (writes_codes && overlap(codes, nc, scales, ns)) return bad("two outputs overlap");
    const Tensor *all = tensors.begin();
    const uint64_t len = columns * e;
    for (size_t i = 0; i < tensors.size(); ++i) {
        const uint64_t whole = (rows - 1) * all[i].stride * e + len;
        if ((all[i].out || writes_codes) && (overlap(all[i].p, whole, codes, nc) || overlap(all[i].p, whole, scales, ns)))
            return bad("what is kept overlaps another tensor");
        for (size_t j = 0; j < i; ++j) {
            if (!all[i].out && !all[j].out) continue;
            if (all[i].out != all[j].out && all[i].p == all[j].p && all[i].stride == all[j].stride) continue;   // in place
            if (rows_overlap(all[i].p, all[i].stride * e, len, all[j].p, all[j].stride * e, len, rows))
                return bad(all[i].out && all[j].out ? "two outputs overlap" : "an output overlaps an input");
        }
    }
    return BF16OPT_OK;
}

template <bool ALIGNED, class K>
int start(K kernel, Args a, cudaStream_t stream) {
    if (sm_count() < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "glu: no CUDA device");
    // threads along a row (whole runs; whole warps where a warp has one row), in pieces of up to a CTA's
    const uint32_t quantum = ALIGNED ? 4 : 32;
    const uint32_t along = (a.runs * 4 + quantum - 1) / quantum * quantum;
    a.blocks = (along + kThreads - 1) / kThreads;
    a.width = (along / quantum + a.blocks - 1) / a.blocks * quantum;
    a.deep = (uint32_t)std::min<uint64_t>(kThreads / a.width, a.rows);
    Launch l{0, (a.width * a.deep + 31) / 32 * 32, 0, stream, 1, true};
    int fit = 0;   // as many as the device holds at once: each walks on
    cudaError_t e = clusters_that_fit(l, kernel, fit);
    if (e != cudaSuccess) return fail_cuda(e, "glu occupancy");
    const uint64_t groups = (a.rows + a.deep - 1) / a.deep;
    l.grid = (unsigned)std::min<uint64_t>(groups, std::max(1u, fit / a.blocks)) * a.blocks;
    l.cluster = 0;   // (CTAs start faster without the attribute)
    e = launch(l, kernel, a);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "glu kernel launch");
}

// Whether every row of these tensors begins on 16 bytes.
bool vectors(int type, std::initializer_list<Tensor> tensors) {
    uint64_t bits = 0;
    for (const Tensor &t : tensors) bits |= (uintptr_t)t.p | t.stride * type_bytes(type);
    return bits % 16 == 0;
}

template <class F>
int by_type(int type, bool vector, F &&f) {
    if (type == BF16OPT_TYPE_BF16) return vector ? f(__nv_bfloat16(), std::true_type()) : f(__nv_bfloat16(), std::false_type());
    return vector ? f(float(), std::true_type()) : f(float(), std::false_type());
}
template <class F>
int by_act(int act, bool gated, F &&f) {
    using Silu = std::integral_constant<int, BF16OPT_GLU_SILU>;
    using Gelu = std::integral_constant<int, BF16OPT_GLU_GELU>;
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (act == BF16OPT_GLU_SILU) return gated ? f(Silu(), Two()) : f(Silu(), One());
    return gated ? f(Gelu(), Two()) : f(Gelu(), One());
}

int pack(const bf16opt_pack_t *d, const void *x, uint64_t x_stride, uint8_t *codes, uint8_t *scales, bool back, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    if (!d) return bad("the descriptor is NULL");
    bool skip;
    const Tensor t = {x, x_stride, back};
    const int rc = check(d->rows, d->columns, d->type, 1, {t}, codes, scales, !back, skip);
    if (rc != BF16OPT_OK || skip) return rc;
    if (!codes || !scales) return bad("a pointer is NULL");
    Args a = {};
    a.rows = d->rows, a.columns = d->columns, a.runs = (d->columns + kRun - 1) / kRun;
    a.codes = codes, a.scales = scales;
    if (back) a.out[0] = const_cast<void *>(x), a.out_stride[0] = x_stride;
    else a.x[0] = {x, x_stride};
    return by_type(d->type, vectors(d->type, {t}), [&](auto zero, auto v) {
        using T = decltype(zero);
        constexpr bool V = decltype(v)::value;
        return back ? start<V>(k_backward<T, V, 1, -1>, a, (cudaStream_t)stream) : start<V>(k_forward<T, V, 1, -1, true>, a, (cudaStream_t)stream);
    });
}

int check_glu(const bf16opt_glu_t *d) {
    if (!d) return bad("the descriptor is NULL");
    if (d->act != BF16OPT_GLU_SILU && d->act != BF16OPT_GLU_GELU) return bad("unknown activation");
    if (d->gated != 0 && d->gated != 1) return bad("gated must be 0 or 1");
    return BF16OPT_OK;
}

int forward(const bf16opt_glu_t *d, Tensor gate, Tensor up, Tensor h, uint8_t *codes, uint8_t *scales, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check_glu(d);
    if (rc != BF16OPT_OK) return rc;
    if (!d->gated && up.p) return bad("up must be NULL without a gate");
    if (!codes != !scales) return bad("codes and scales go together");
    bool skip;
    rc = d->gated ? check(d->rows, d->columns, d->type, 2, {gate, up, h}, codes, scales, codes != nullptr, skip)
                  : check(d->rows, d->columns, d->type, 1, {gate, h}, codes, scales, codes != nullptr, skip);
    if (rc != BF16OPT_OK || skip) return rc;
    Args a = {};
    a.rows = d->rows, a.columns = d->columns, a.runs = (d->columns + kRun - 1) / kRun;
    a.codes = codes, a.scales = scales;
    a.x[0] = {gate.p, gate.stride}, a.x[1] = {up.p, up.stride};
    a.out[0] = const_cast<void *>(h.p), a.out_stride[0] = h.stride;
    const bool v = d->gated ? vectors(d->type, {gate, up, h}) : vectors(d->type, {gate, h});
    return by_type(d->type, v, [&](auto zero, auto v) {
        using T = decltype(zero);
        constexpr bool V = decltype(v)::value;
        return by_act(d->act, d->gated, [&](auto act, auto parts) {
            constexpr int A = decltype(act)::value, P = decltype(parts)::value;
            return codes ? start<V>(k_forward<T, V, P, A, true>, a, (cudaStream_t)stream) : start<V>(k_forward<T, V, P, A, false>, a, (cudaStream_t)stream);
        });
    });
}

int backward(const bf16opt_glu_t *d, Tensor dh, const uint8_t *codes, const uint8_t *scales, Tensor dgate, Tensor dup, Tensor h, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check_glu(d);
    if (rc != BF16OPT_OK) return rc;
    if (!d->gated && dup.p) return bad("dup must be NULL without a gate");
    bool skip;
    const uint32_t parts = d->gated ? 2 : 1;
    auto checked = [&](std::initializer_list<Tensor> t) { return check(d->rows, d->columns, d->type, parts, t, codes, scales, false, skip); };
    rc = d->gated ? (h.p ? checked({dh, dgate, dup, h}) : checked({dh, dgate, dup})) : (h.p ? checked({dh, dgate, h}) : checked({dh, dgate}));
    if (rc != BF16OPT_OK || skip) return rc;
    if (!codes || !scales) return bad("a pointer is NULL");
    Args a = {};
    a.rows = d->rows, a.columns = d->columns, a.runs = (d->columns + kRun - 1) / kRun;
    a.codes = const_cast<uint8_t *>(codes), a.scales = const_cast<uint8_t *>(scales);
    a.x[0] = {dh.p, dh.stride};
    const Tensor *outs[3] = {&dgate, &dup, &h};
    bool v = vectors(d->type, {dh});
    for (int i = 0; i < 3; ++i) {
        a.out[i] = const_cast<void *>(outs[i]->p), a.out_stride[i] = outs[i]->stride;
        if (outs[i]->p) v = v && vectors(d->type, {*outs[i]});
    }
    return by_type(d->type, v, [&](auto zero, auto v) {
        using T = decltype(zero);
        constexpr bool V = decltype(v)::value;
        return by_act(d->act, d->gated, [&](auto act, auto parts) {
            return start<V>(k_backward<T, V, decltype(parts)::value, decltype(act)::value>, a, (cudaStream_t)stream);
        });
    });
}

}  // namespace
}  // namespace bf16ops

extern "C" int bf16opt_pack(const bf16opt_pack_t *d, const void *x, uint64_t x_stride, uint8_t *codes, uint8_t *scales, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::pack(d, x, x_stride, codes, scales, false, stream); });
}

extern "C" int bf16opt_unpack(const bf16opt_pack_t *d, const uint8_t *codes, const uint8_t *scales, void *x, uint64_t x_stride, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::pack(d, x, x_stride, const_cast<uint8_t *>(codes), const_cast<uint8_t *>(scales), true, stream); });
}

extern "C" int bf16opt_glu_forward(const bf16opt_glu_t *d, const void *gate, uint64_t gate_stride, const void *up, uint64_t up_stride,
                                   void *h, uint64_t h_stride, uint8_t *codes, uint8_t *scales, void *stream) {
    return bf16ops::guarded([&] {
        return bf16ops::forward(d, {gate, gate_stride, false}, {up, up_stride, false}, {h, h_stride, true}, codes, scales, stream);
    });
}

extern "C" int bf16opt_glu_backward(const bf16opt_glu_t *d, const void *dh, uint64_t dh_stride, const uint8_t *codes,
                                    const uint8_t *scales, void *dgate, uint64_t dgate_stride, void *dup, uint64_t dup_stride,
                                    void *h, uint64_t h_stride, void *stream) {
    return bf16ops::guarded([&] {
        return bf16ops::backward(d, {dh, dh_stride, false}, codes, scales, {dgate, dgate_stride, true}, {dup, dup_stride, true},
                                 {h, h_stride, true}, stream);
    });
}
