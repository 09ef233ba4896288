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
    uint32_t columns, runs;
};

// ------------------------------------------------------------------ a run's scale

// The scale's byte for a run whose largest finite magnitude has the bits `m`: its exponent less 8, one
// more where the fraction is above 1.75 (448 = 1.75 * 2^8), and no less than 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
    const uint32_t e = (m + 0x1fffffu) >> 23;
    return e > 8 ? e - 8 : 0u;
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 1u << 22); }   // 2^(byte - 127)
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// What would be rounded to 2^128 is kept as the number below it, 1.875 2^127; an infinity as NaN.
constexpr float kTooLarge = 0x1.fp127f;
__device__ __forceinline__ float holdable(float x) {
    return fabsf(x) < kTooLarge ? x : fabsf(x) < INFINITY ? copysignf(0x1.ep127f, x) : NAN;
}

// Two floats to e4m3, the first in the low byte.  (NaN stays NaN; an infinity is made one before.)
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_codes(uint32_t two) {   // exact in fp16
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float2 f;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

// ------------------------------------------------------------------ the activation

// sigmoid(y) and 1 - sigmoid(y): e = exp(-y), 1 / (1 + e) and e / (1 + e), each exact where the other cancels.  The
// exponent stops at 2^127: 1 / (1 + 2^127) is flushed to 0, and 0 e is 0.
__device__ __forceinline__ void sigmoids(float y, float &s, float &rest) {
    const float x = y * -kLog2e;
    const float e = ex2(x > 127.f ? 127.f : x);   // (a NaN stays one)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    rest = e * s;
}

// act(g) = g sigmoid(y), y = g (silu) or 2 sqrt(2 / pi) (g + 0.044715 g^3) (gelu: (1 + tanh(y / 2)) / 2 = sigmoid(y)), and
// act'(g) = sigmoid(y) + g sigmoid(y) (1 - sigmoid(y)) y'.  Beyond +-64 the sigmoid is 0 or 1, and g^3 is not formed.
template <int ACT>
__device__ __forceinline__ float activate(float g, float &slope) {
    constexpr float kRoot = 1.59576912160573071f;   // 2 sqrt(2 / pi)
    float y = g, c = g, dy = 1.f;
    if (ACT == BF16OPT_GLU_GELU) {
        c = g > 64.f ? 64.f : g < -64.f ? -64.f : g;
        const float q = c * c;
        y = kRoot * c * fmaf(0.044715f, q, 1.f);
        dy = kRoot * fmaf(3.f * 0.044715f, q, 1.f);
    }
    float s, rest;
    sigmoids(y, s, rest);
    slope = fmaf(c * dy, s * rest, s);
    return g * s;
}

// ------------------------------------------------------------------ eight columns of a thread

// VECTOR: eight neighbours, four lanes to a run; rows and their starts are multiples of 16 bytes.
// Otherwise columns lane, lane + 32, ..: a run is a warp's, whatever the alignment.
template <class T, bool VECTOR>
struct Eight {
    // column of element i
    __device__ __forceinline__ static uint32_t column(uint32_t first, int i) { return VECTOR ? first + i : first + 32 * i; }
    __device__ __forceinline__ static void load(const T *row, uint32_t first, uint32_t columns, float (&f)[8]) {
        if (VECTOR && first + 8 <= columns) {
            const uint4 *v = reinterpret_cast<const uint4 *>(row + first);
            if constexpr (sizeof(T) == 2) {
                Vec<T>::unpack(__ldcs(v), f);
            } else {
                float a[4], b[4];
                const uint4 x = __ldcs(v), y = __ldcs(v + 1);
                Vec<T>::unpack(x, a), Vec<T>::unpack(y, b);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = column(first, i) < columns ? to_f32(row[column(first, i)]) : 0.f;
        }
    }
    __device__ __forceinline__ static void store(T *row, uint32_t first, uint32_t columns, const float (&f)[8]) {
        if (VECTOR && first + 8 <= columns) {
            uint4 *v = reinterpret_cast<uint4 *>(row + first);
            if constexpr (sizeof(T) == 2) {
                __stcs(v, Vec<T>::pack(f));
            } else {
                __stcs(v, Vec<T>::pack({f[0], f[1], f[2], f[3]}));
                __stcs(v + 1, Vec<T>::pack({f[4], f[5], f[6], f[7]}));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (column(first, i) < columns) from_f32(row[column(first, i)], f[i]);
        }
    }
};

// Keeps the warp's (or its quads') values.  Every lane of the warp takes part; `there`: the lane's columns lie
// within the row's runs.
template <bool VECTOR>
__device__ __forceinline__ void keep(const float (&f)[8], uint8_t *codes, uint8_t *scales, uint32_t first, uint32_t runs, bool there) {
    if (VECTOR) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));   // NaN passed over
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = f[i];
        if (__any_sync(0xffffffffu, m >= kTooLarge)) {   // the largest finite one, NaN for the infinite
            m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (fabsf(f[i]) < INFINITY) m = fmaxf(m, fabsf(f[i]));
                x[i] = holdable(f[i]);
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        }
        if (!there) return;
        const uint32_t byte = scale_byte(__float_as_uint(m));
        const float inv = inverse_scale(byte);
        uint2 c;
        c.x = to_codes(x[0] * inv, x[1] * inv) | to_codes(x[2] * inv, x[3] * inv) << 16;
        c.y = to_codes(x[4] * inv, x[5] * inv) | to_codes(x[6] * inv, x[7] * inv) << 16;
        *reinterpret_cast<uint2 *>(codes + first) = c;
        if ((first & (kRun - 1)) == 0) scales[first / kRun] = (uint8_t)byte;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool fine = fabsf(f[i]) < INFINITY;
            const float m = warp_max(fine ? fabsf(f[i]) : 0.f);
            const uint32_t byte = scale_byte(__float_as_uint(m));
            const uint32_t run = first / kRun + i;
            if (run < runs) {
                codes[first + 32 * i] = (uint8_t)to_codes(holdable(f[i]) * inverse_scale(byte), 0.f);
                if ((first & (kRun - 1)) == 0) scales[run] = (uint8_t)byte;
            }
        }
    }
}

template <bool VECTOR>
__device__ __forceinline__ void read(const uint8_t *codes, const uint8_t *scales, uint32_t first, uint32_t runs, float (&f)[8]) {
    if (VECTOR) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2 *>(codes + first));
        const float s = scale_of(scales[first / kRun]);
        const uint32_t two[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = mul2(from_codes(two[i]), both(s));
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t run = first / kRun + i;
            f[i] = run < runs ? from_codes(codes[first + 32 * i]).x * scale_of(scales[run]) : 0.f;
        }
    }
}

// ------------------------------------------------------------------ the kernels

// A warp takes 256 columns of a row at a time.  PARTS: 1 or 2 of what is kept; ACT < 0: nothing but keeping or reading.
template <class T, bool VECTOR, int PARTS, int ACT, bool KEEP>
__global__ void __launch_bounds__(kThreads) k_forward(const Args a) {
    using E = Eight<T, VECTOR>;
    pdl_enter();
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t spans = (a.columns + 255) / 256;
    const uint64_t n = a.rows * spans, step = (uint64_t)gridDim.x * (kThreads / 32);
    for (uint64_t w = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; w < n; w += step) {
        const uint64_t row = w / spans;
        const uint32_t first = (uint32_t)(w - row * spans) * 256 + (VECTOR ? lane * 8 : lane);
        float f[PARTS][8];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) E::load(reinterpret_cast<const T *>(a.x[p].p) + row * a.x[p].stride, first, a.columns, f[p]);
        if (ACT >= 0) {
            float h[8], slope;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = activate<ACT>(f[0][i], slope);
                if (PARTS > 1) h[i] *= f[PARTS - 1][i];
            }
            E::store(reinterpret_cast<T *>(a.out[0]) + row * a.out_stride[0], first, a.columns, h);
        }
        if (KEEP) {
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const uint64_t at = (p * a.rows + row) * a.runs;
                keep<VECTOR>(f[p], a.codes + at * kRun, a.scales + at, first, a.runs, first < a.runs * kRun);
            }
        }
    }
    pdl_leave();
}

template <class T, bool VECTOR, int PARTS, int ACT>
__global__ void __launch_bounds__(kThreads) k_backward(const Args a) {
    using E = Eight<T, VECTOR>;
    pdl_enter();
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t spans = (a.columns + 255) / 256;
    const uint64_t n = a.rows * spans, step = (uint64_t)gridDim.x * (kThreads / 32);
    for (uint64_t w = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; w < n; w += step) {
        const uint64_t row = w / spans;
        const uint32_t first = (uint32_t)(w - row * spans) * 256 + (VECTOR ? lane * 8 : lane);
        if (first >= a.runs * kRun) continue;
        float f[PARTS][8], dh[8];
        if (ACT >= 0) E::load(reinterpret_cast<const T *>(a.x[0].p) + row * a.x[0].stride, first, a.columns, dh);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const uint64_t at = (p * a.rows + row) * a.runs;
            read<VECTOR>(a.codes + at * kRun, a.scales + at, first, a.runs, f[p]);
        }
        auto put = [&](int i, const float (&v)[8]) { E::store(reinterpret_cast<T *>(a.out[i]) + row * a.out_stride[i], first, a.columns, v); };
        if constexpr (ACT < 0) {
            put(0, f[0]);
        } else {
            float dg[8], du[8], h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float slope;
                const float act = activate<ACT>(f[0][i], slope);
                dg[i] = dh[i] * slope;
                h[i] = act;
                if (PARTS > 1) {
                    dg[i] *= f[PARTS - 1][i];
                    du[i] = dh[i] * act;
                    h[i] *= f[PARTS - 1][i];
                }
            }
            put(0, dg);
            if (PARTS > 1) put(1, du);
            if (a.out[2]) put(2, h);
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
    if (!span_bytes(rows, runs * kRun * parts, runs * kRun * parts, 1, bytes) || rows >= (1ull << 40)) return bad("the sizes overflow");
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

template <class K>
int start(K kernel, const Args &a, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "glu: no CUDA device");
    const uint64_t warps = a.rows * ((a.columns + 255) / 256), ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    const cudaError_t e = launch(Launch{(unsigned)std::min<uint64_t>(ctas, (uint64_t)sms * 8), kThreads, 0, stream, 0, true}, kernel, a);
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
        return back ? start(k_backward<T, V, 1, -1>, a, (cudaStream_t)stream) : start(k_forward<T, V, 1, -1, true>, a, (cudaStream_t)stream);
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
            return codes ? start(k_forward<T, V, P, A, true>, a, (cudaStream_t)stream) : start(k_forward<T, V, P, A, false>, a, (cudaStream_t)stream);
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
            return start(k_backward<T, V, decltype(parts)::value, decltype(act)::value>, a, (cudaStream_t)stream);
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
