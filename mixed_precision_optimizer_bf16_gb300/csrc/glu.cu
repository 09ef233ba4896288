// glu.cu -- activations kept in 8 bits (bf16opt_pack, bf16opt_unpack) and a feed-forward block's
// activation that keeps its inputs so (bf16opt_glu_*), of include/bf16opt.h.
//
// Everything here is element by element but for a run's largest magnitude, and is bound by its bytes: per
// element of bf16, forward 2 (read) + 1 + 1/32 (kept) for gate and for up and 2 for h;
// backward 2 (dh) + the same kept ones, and 2 for each gradient.
//
// A scale is a power of two, so dividing by it is exact and a code depends on nothing but the
// element and its run's largest: no rounding but the one to e4m3 (half a step of three bits: 2^-4
// relative at most, down to 2^-14 of the run's largest or so).
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
// sigmoid(y)); act'(g) = s + g y' s (1 - s).  1 - s as a difference is off by 2^-24, which times g y' is about |y| 2^-24 of
// act'.  From |g| = 64 on gelu's sigmoid is 0 or 1, and g^2 stops growing.  (NaN goes through g.)
template <int ACT>
__device__ __forceinline__ float2 activate(float2 g, float2 &slope) {
    constexpr float kA = 1.59576912160573071f, kB = 0.044715f * kA;
    float2 y = g, dy = both(1.f);
    if (ACT == BF16OPT_GLU_GELU) {
        float2 q = mul2(g, g);
        q = make_float2(fminf(q.x, 4096.f), fminf(q.y, 4096.f));
        y = mul2(g, fma2(q, both(kB), both(kA)));
        dy = fma2(q, both(3.f * kB), both(kA));
    }
    const float2 x = mul2(y, both(-kLog2e)), t = add2(make_float2(ex2(x.x), ex2(x.y)), both(1.f));
    const float2 s = make_float2(reciprocal(t.x), reciprocal(t.y));
    float2 w = mul2(s, fma2(s, both(-1.f), both(1.f)));
    if (ACT == BF16OPT_GLU_GELU) w = mul2(w, dy);
    slope = fma2(g, w, s);
    return mul2(g, s);
}

// ------------------------------------------------------------------ eight columns of a thread

// VECTOR: eight neighbours from `first`, four lanes to a run; rows and their starts are multiples of 16 bytes.
// Otherwise columns first, first + 32, ..: a run is a warp's, whatever the alignment.
template <class T, bool VECTOR>
struct Eight {
    static constexpr int W = sizeof(T) / 2;
    union {
        uint4 v[W];
        T e[8];
    };
    __device__ __forceinline__ Eight() {}
    __device__ __forceinline__ static uint32_t column(uint32_t first, int i) { return VECTOR ? first + i : first + 32 * i; }
    __device__ __forceinline__ void load(const T *row, uint32_t first, uint32_t columns) {
        if (VECTOR && first + 8 <= columns) {
#pragma unroll
            for (int w = 0; w < W; ++w) v[w] = __ldcs(reinterpret_cast<const uint4 *>(row + first) + w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (column(first, i) < columns) e[i] = row[column(first, i)];
                else from_f32(e[i], 0.f);
            }
        }
    }
    __device__ __forceinline__ void store(T *row, uint32_t first, uint32_t columns) const {
        if (VECTOR && first + 8 <= columns) {
#pragma unroll
            for (int w = 0; w < W; ++w) __stcs(reinterpret_cast<uint4 *>(row + first) + w, v[w]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (column(first, i) < columns) row[column(first, i)] = e[i];
        }
    }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        if constexpr (sizeof(T) == 2) {
            f[0] = make_float2(bf16_lo(v[0].x), bf16_hi(v[0].x)), f[1] = make_float2(bf16_lo(v[0].y), bf16_hi(v[0].y));
            f[2] = make_float2(bf16_lo(v[0].z), bf16_hi(v[0].z)), f[3] = make_float2(bf16_lo(v[0].w), bf16_hi(v[0].w));
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                f[2 * w] = make_float2(__uint_as_float(v[w].x), __uint_as_float(v[w].y));
                f[2 * w + 1] = make_float2(__uint_as_float(v[w].z), __uint_as_float(v[w].w));
            }
        }
    }
    __device__ __forceinline__ void pack(const float2 (&f)[4]) {
        if constexpr (sizeof(T) == 2) {
            v[0] = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
        } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
                v[w] = make_uint4(__float_as_uint(f[2 * w].x), __float_as_uint(f[2 * w].y), __float_as_uint(f[2 * w + 1].x), __float_as_uint(f[2 * w + 1].y));
        }
    }
};

// A thread's columns, and the rows that it walks down: the CTA's first one, then every `step`-th.
struct Place {
    uint32_t first, run;   // first column; its run in the row
    bool there;            // the thread has columns within the row's runs
    uint32_t row, step;
};
template <bool VECTOR>
__device__ __forceinline__ Place place_of(const Args &a) {
    const uint32_t group = blockIdx.x / a.blocks, block = blockIdx.x - group * a.blocks;
    const uint32_t slot = threadIdx.x / a.width, i = block * a.width + (threadIdx.x - slot * a.width);
    Place p;
    p.first = VECTOR ? i * 8 : i / 32 * 256 + i % 32;
    p.run = p.first / kRun;
    p.there = p.first < a.runs * kRun && slot < a.deep;
    p.row = group * a.deep + slot;
    p.step = gridDim.x / a.blocks * a.deep;
    return p;
}

// Keeps the thread's columns of one row.  Every lane of the warp takes part; `there`: it has any.
template <bool VECTOR, int PARTS>
__device__ __forceinline__ void keep(const Args &a, const float2 (&f)[PARTS][4], uint8_t *codes, uint8_t *scales, const Place &p, bool there) {
    if (VECTOR) {
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
    } else {
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = i & 1 ? f[k][i / 2].y : f[k][i / 2].x;
                const uint32_t byte = scale_byte(warp_max(fabsf(x) < INFINITY ? fabsf(x) : 0.f));
                if (there && p.run + i < a.runs) {
                    codes[k * a.rows * a.runs * kRun + 32 * i] = (uint8_t)to_codes(holdable(x) * inverse_scale(byte), 0.f);
                    if ((threadIdx.x & 31) == 0) scales[k * a.rows * a.runs + i] = (uint8_t)byte;
                }
            }
        }
    }
}

// What was kept, on its way: VECTOR: eight codes and their scale.
template <bool VECTOR>
struct Kept {
    uint2 c;
    uint32_t byte;
    uint8_t codes[VECTOR ? 1 : 8], bytes[VECTOR ? 1 : 8];
    __device__ __forceinline__ void load(const uint8_t *from, const uint8_t *scale, uint32_t run, uint32_t runs) {
        if (VECTOR) {
            c = __ldcs(reinterpret_cast<const uint2 *>(from));
            byte = *scale;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                codes[VECTOR ? 0 : i] = run + i < runs ? from[32 * i] : (uint8_t)0;
                bytes[VECTOR ? 0 : i] = run + i < runs ? scale[i] : (uint8_t)0;
            }
        }
    }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        if (VECTOR) {
            const float2 s = both(scale_of(byte));
            f[0] = mul2(from_codes(c.x & 0xffffu), s), f[1] = mul2(from_codes(c.x >> 16), s);
            f[2] = mul2(from_codes(c.y & 0xffffu), s), f[3] = mul2(from_codes(c.y >> 16), s);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = VECTOR ? 0 : 2 * i, y = VECTOR ? 0 : 2 * i + 1;
                f[i] = mul2(from_codes(codes[x] | (uint32_t)codes[y] << 8), make_float2(scale_of(bytes[x]), scale_of(bytes[y])));
            }
        }
    }
};

// ------------------------------------------------------------------ the kernels

// A thread has its columns and walks down the rows with them, `U` rows at a time, the next ones on their way while it
// works on these: addresses only go on by a stride.  U: so many that 32 bytes or so of each thread are on their way.

// PARTS: 1 or 2 of what is kept; ACT < 0: nothing but keeping or reading.
template <class T, bool VECTOR, int PARTS, int ACT, bool KEEP>
__global__ void __launch_bounds__(kThreads) k_forward(const Args a) {
    constexpr int U = sizeof(T) == 2 && PARTS == 1 && VECTOR ? 2 : 1;
    using E = Eight<T, VECTOR>;
    pdl_enter();
    const Place p = place_of<VECTOR>(a);
    const T *x[PARTS];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) x[k] = reinterpret_cast<const T *>(a.x[k].p) + p.row * a.x[k].stride;
    T *h = reinterpret_cast<T *>(a.out[0]) + p.row * a.out_stride[0];
    uint8_t *codes = a.codes + (uint64_t)p.row * a.runs * kRun + p.first, *scales = a.scales + (uint64_t)p.row * a.runs + p.run;
    E next[U][PARTS];
    auto ask = [&](uint32_t row) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                next[u][k].load(x[k], p.there && row + u * p.step < a.rows ? p.first : a.columns, a.columns);
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
            for (int k = 0; k < PARTS; ++k) next[u][k].unpack(f[u][k]);
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
                if (there) e.store(h, p.first, a.columns);
                h += p.step * a.out_stride[0];
            }
            if (KEEP) {
                keep<VECTOR, PARTS>(a, f[u], codes, scales, p, there);
                codes += (uint64_t)p.step * a.runs * kRun, scales += (uint64_t)p.step * a.runs;
            }
        }
    }
    pdl_leave();
}

template <class T, bool VECTOR, int PARTS, int ACT>
__global__ void __launch_bounds__(kThreads, VECTOR ? 4 : 2) k_backward(const Args a) {
    constexpr int U = ACT < 0 && VECTOR ? 4 : 1;
    using E = Eight<T, VECTOR>;
    pdl_enter();
    const Place p = place_of<VECTOR>(a);
    if (!p.there) return;
    const T *x = reinterpret_cast<const T *>(a.x[0].p) + p.row * a.x[0].stride;
    const uint8_t *codes = a.codes + (uint64_t)p.row * a.runs * kRun + p.first, *scales = a.scales + (uint64_t)p.row * a.runs + p.run;
    constexpr int kOuts = ACT < 0 ? 1 : 3;
    T *out[kOuts];
#pragma unroll
    for (int i = 0; i < kOuts; ++i) out[i] = reinterpret_cast<T *>(a.out[i]) + p.row * a.out_stride[i];
    E next;
    Kept<VECTOR> kept[U][PARTS];
    auto ask = [&](uint32_t row) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row + u * p.step < a.rows) {
                if (ACT >= 0) next.load(x, p.first, a.columns);
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
                    kept[u][k].load(codes + k * a.rows * a.runs * kRun, scales + k * a.rows * a.runs, p.run, a.runs);
            }
            if (ACT >= 0) x += p.step * a.x[0].stride;
            codes += (uint64_t)p.step * a.runs * kRun, scales += (uint64_t)p.step * a.runs;
        }
    };
    ask(p.row);
    for (uint32_t row = p.row; row < a.rows; row += U * p.step) {
        float2 f[U][PARTS][4], dh[4];
        if (ACT >= 0) next.unpack(dh);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) kept[u][k].unpack(f[u][k]);
        ask(row + U * p.step);
        auto put = [&](int i, const float2 (&v)[4]) {
            E e;
            e.pack(v);
            e.store(out[i], p.first, a.columns);
        };
        if constexpr (ACT < 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (row + u * p.step < a.rows) put(0, f[u][0]);
                out[0] += p.step * a.out_stride[0];
            }
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
            put(0, dg);
            if (PARTS > 1) put(1, du);
            if (a.out[2]) put(2, h);
#pragma unroll
            for (int i = 0; i < kOuts; ++i) out[i] += p.step * a.out_stride[i];
        }
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

template <bool VECTOR, class K>
int start(K kernel, Args a, cudaStream_t stream) {
    if (sm_count() < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "glu: no CUDA device");
    // threads along a row (whole runs, whole warps where a run is a warp's), in pieces of up to a CTA's
    const uint32_t quantum = VECTOR ? 4 : 32;
    const uint32_t along = VECTOR ? a.runs * 4 : (a.columns + 255) / 256 * 32;
    a.blocks = (along + kThreads - 1) / kThreads;
    a.width = (along / quantum + a.blocks - 1) / a.blocks * quantum;
    a.deep = (uint32_t)std::min<uint64_t>(kThreads / a.width, a.rows);
    Launch l{0, (a.width * a.deep + 31) / 32 * 32, 0, stream, 1, true};
    int fit = 0;   // as many as the device holds at once: each walks on
    cudaError_t e = clusters_that_fit(l, kernel, fit);
    if (e != cudaSuccess) return fail_cuda(e, "glu occupancy");
    const uint64_t groups = (a.rows + a.deep - 1) / a.deep;
    l.grid = (unsigned)std::min<uint64_t>(groups, std::max(1u, fit / a.blocks)) * a.blocks;
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
