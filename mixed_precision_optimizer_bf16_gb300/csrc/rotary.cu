// rotary.cu -- rotary positions, forward and backward (bf16opt_rotary of include/bf16opt.h).
//
// Every element is read once and written once, which is what bounds the operator; q and k go
// in one launch.  A thread has one place in the head (a vector of elements and, in the half layout, its
// partners') and walks over tokens and heads with it, so its frequencies stay in registers
// and an angle's sine and cosine are computed once per token for all the heads that it turns.
//
// The angle: position times frequency, both whole numbers (2^-64 turns), wraps around
// at whole turns by itself; what is left, in (-1/2, 1/2] turns, goes to FP32.
#include "ops_common.cuh"

namespace bf16ops {
namespace {

constexpr int kThreads = 256;

struct Place {
    const void *in;
    void *out;
    uint64_t in_b, in_t, in_h, out_b, out_t, out_h;   // elements between batches, tokens, heads
};

struct Args {
    Place q, k;
    uint64_t tokens, seq;       // tokens: batch * seq
    const void *positions;
    uint64_t positions_stride;
    int64_t offset;
    int positions_type;
    uint32_t heads, all_heads;  // of q; of q and k
    uint32_t dim, turned;
    uint32_t units;             // threads of a head: the ones that turn, then the ones that copy
    uint32_t turning;           // of them turning
    uint32_t lanes;             // heads side by side in a CTA
    uint32_t group;             // tokens side by side in a CTA
    float scale;
    uint32_t inverse;
    uint64_t turns[BF16OPT_ROTARY_MAX_DIM / 2];   // 2^-64 turns per position
};

// N elements at p as floats, and back.  WIDE: as one access.
template <class T, int N, bool WIDE>
__device__ __forceinline__ void load_n(const T *p, float (&f)[N]) {
    if constexpr (WIDE && N * sizeof(T) == 16) {
        Vec<T>::unpack(__ldcs(reinterpret_cast<const uint4 *>(p)), f);
    } else if constexpr (WIDE && N * sizeof(T) == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        if constexpr (sizeof(T) == 2) f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
        else f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
    } else if constexpr (WIDE && N * sizeof(T) == 4 && sizeof(T) == 2) {
        const uint32_t v = __ldcs(reinterpret_cast<const unsigned int *>(p));
        f[0] = bf16_lo(v), f[1] = bf16_hi(v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32(p[i]);
    }
}
template <class T, int N, bool WIDE>
__device__ __forceinline__ void store_n(T *p, const float (&f)[N]) {
    if constexpr (WIDE && N * sizeof(T) == 16) {
        __stcs(reinterpret_cast<uint4 *>(p), Vec<T>::pack(f));
    } else if constexpr (WIDE && N * sizeof(T) == 8) {
        uint2 v;
        if constexpr (sizeof(T) == 2) v = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
        else v = make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1]));
        __stcs(reinterpret_cast<uint2 *>(p), v);
    } else if constexpr (WIDE && N * sizeof(T) == 4 && sizeof(T) == 2) {
        __stcs(reinterpret_cast<unsigned int *>(p), pack_bf16(f[0], f[1]));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) from_f32(p[i], f[i]);
    }
}

template <class T, int N, bool WIDE>
__device__ __forceinline__ void copy_n(T *to, const T *from) {
    if constexpr (WIDE && N * sizeof(T) == 16) {
        __stcs(reinterpret_cast<uint4 *>(to), __ldcs(reinterpret_cast<const uint4 *>(from)));
    } else if constexpr (WIDE && N * sizeof(T) == 8) {
        __stcs(reinterpret_cast<uint2 *>(to), __ldcs(reinterpret_cast<const uint2 *>(from)));
    } else if constexpr (WIDE && N * sizeof(T) == 4 && sizeof(T) == 2) {
        __stcs(reinterpret_cast<unsigned int *>(to), __ldcs(reinterpret_cast<const unsigned int *>(from)));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = from[i];
    }
}

// (Spelt out, so that a result does not depend on the variant that computes it.)
__device__ __forceinline__ void turned_pair(float a, float b, float c, float s, float &u, float &v) {
    u = fmaf(-b, s, __fmul_rn(a, c));
    v = fmaf(a, s, __fmul_rn(b, c));
}

// HALF: a thread turns N pairs (i, i + turned / 2); else N / 2 pairs of neighbours.
template <class T, int N, bool WIDE, bool HALF>
__global__ void __launch_bounds__(kThreads) k_rotary(const Args a) {
    constexpr int P = HALF ? N : N / 2;   // pairs of a thread
    pdl_enter();
    const uint32_t per_token = a.units * a.lanes;
    const uint32_t slot = threadIdx.x / per_token, left = threadIdx.x - slot * per_token;
    const uint32_t lane = left / a.units, unit = left - lane * a.units;
    if (slot >= a.group) return;
    const bool turn = unit < a.turning;
    const uint32_t at = turn ? unit * N : a.turned + (unit - a.turning) * N;   // the thread's first element
    uint64_t turns[P];
#pragma unroll
    for (int i = 0; i < P; ++i) turns[i] = turn ? a.turns[unit * P + i] : 0;
    for (uint64_t token = (uint64_t)blockIdx.x * a.group + slot; token < a.tokens; token += (uint64_t)gridDim.x * a.group) {
        const uint64_t b = a.tokens == a.seq ? 0 : token / a.seq, t = token - b * a.seq;
        float cs[P], sn[P];
        if (turn) {
            const int64_t pos = (a.positions ? load_index(a.positions, a.positions_type, b * a.positions_stride + t) : (int64_t)t);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int32_t part = (int32_t)(((uint64_t)pos + (uint64_t)a.offset) * turns[i] >> 32);   // of a turn, in 2^-32
                sincospif((float)part * 0x1p-31f, &sn[i], &cs[i]);
                cs[i] *= a.scale;
                sn[i] *= a.inverse ? -a.scale : a.scale;
            }
        }
        for (uint32_t head = lane; head < a.all_heads; head += a.lanes) {
            const bool is_q = head < a.heads;
            const Place &pl = is_q ? a.q : a.k;
            const uint32_t h = is_q ? head : head - a.heads;
            const T *in = reinterpret_cast<const T *>(pl.in) + b * pl.in_b + t * pl.in_t + h * pl.in_h + at;
            T *out = reinterpret_cast<T *>(pl.out) + b * pl.out_b + t * pl.out_t + h * pl.out_h + at;
            if (turn) {
                if constexpr (HALF) {
                    const uint32_t half = a.turned / 2;
                    float x[N], y[N], u[N], v[N];
                    load_n<T, N, WIDE>(in, x);
                    load_n<T, N, WIDE>(in + half, y);
#pragma unroll
                    for (int i = 0; i < N; ++i) turned_pair(x[i], y[i], cs[i], sn[i], u[i], v[i]);
                    store_n<T, N, WIDE>(out, u);
                    store_n<T, N, WIDE>(out + half, v);
                } else {
                    float x[N], u[N];
                    load_n<T, N, WIDE>(in, x);
#pragma unroll
                    for (int i = 0; i < P; ++i) turned_pair(x[2 * i], x[2 * i + 1], cs[i], sn[i], u[2 * i], u[2 * i + 1]);
                    store_n<T, N, WIDE>(out, u);
                }
            } else if (in != out) {
                for (uint32_t i = 0; at + i < a.dim; i += (a.units - a.turning) * N) {
                    if (WIDE || at + i + N <= a.dim) {
                        copy_n<T, N, WIDE>(out + i, in + i);
                    } else {
                        for (uint32_t j = i; at + j < a.dim; ++j) out[j] = in[j];
                    }
                }
            }
        }
    }
    pdl_leave();
}

// ---------------------------------------------------------------------- host

struct Box {   // a tensor [batch, tokens, heads, dim] in bytes
    const void *p;
    uint64_t n[3], s[3], len;
};

uint64_t span(const Box &x, int from = 0) {   // bytes from the first to behind the last, over dimensions `from` and on
    uint64_t n = x.len;
    for (int i = from; i < 3; ++i) n += (x.n[i] - 1) * x.s[i];
    return n;
}

// Whether no element of x is there twice: each dimension steps over all that the ones with smaller strides span.
bool apart(const Box &x) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int i, int j) { return x.s[i] < x.s[j]; });
    uint64_t n = x.len;
    for (int i : order) {
        if (x.n[i] == 1) continue;
        if (x.s[i] < n) return false;
        n += (x.n[i] - 1) * x.s[i];
    }
    return true;
}

// Whether x and y may share a byte: not where their spans are apart, or where at each step of
// a stride that they share (between batches, or between tokens) the rest of them is.
bool may_overlap(const Box &x, const Box &y) {
    if (!overlap(x.p, span(x), y.p, span(y))) return false;
    for (int i = 0; i < 2; ++i) {
        const uint64_t m = x.s[i];
        if (m == 0 || m != y.s[i] || (x.n[i] == 1 && y.n[i] == 1)) continue;
        if (i == 1 && x.n[0] > 1 && (x.s[0] % m || y.s[0] % m)) continue;   // whole steps between batches too
        const uint64_t nx = span(x, i + 1), ny = span(y, i + 1);
        const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
        const uint64_t from = b >= a ? (b - a) % m : (m - (a - b) % m) % m;
        if (from >= nx && from + ny <= m) return false;
    }
    return true;
}

bool box(Box &x, const bf16opt_rotary_t *d, const void *p, const uint64_t (&stride)[3], uint32_t heads) {
    const uint64_t e = type_bytes(d->type);
    x.p = p;
    x.n[0] = d->batch, x.n[1] = d->seq, x.n[2] = heads;
    x.len = d->dim * e;
    unsigned __int128 n = x.len;
    for (int i = 0; i < 3; ++i) {
        const unsigned __int128 s = (unsigned __int128)stride[i] * e;
        if (x.n[i] > 1 && s >> 62) return false;
        x.s[i] = x.n[i] > 1 ? (uint64_t)s : 0;   // of one item no stride counts
        n += (unsigned __int128)(x.n[i] - 1) * x.s[i];
    }
    return n >> 62 == 0;
}

bool same(const Box &x, const Box &y) {
    return x.p == y.p && x.s[0] == y.s[0] && x.s[1] == y.s[1] && x.s[2] == y.s[2];
}

template <class T, int N, bool WIDE, bool HALF>
int start(Args &a, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "rotary: no CUDA device");
    const uint32_t width = HALF ? 2 * N : N;   // elements that a thread turns
    a.turning = a.turned / width;
    a.units = a.turning + std::min((a.dim - a.turned + N - 1) / N, (uint32_t)kThreads / 2);   // (at most half the threads turn)
    // heads side by side: a thread takes up to eight heads of a token (its sines serve them all), fewer while the SMs are not full
    uint32_t most = 8;
    while (most > 1 && a.tokens * ((a.all_heads + most - 1) / most) * a.units < (uint64_t)sms * 1024) most /= 2;
    a.lanes = std::min(kThreads / a.units, (a.all_heads + most - 1) / most);
    a.group = kThreads / (a.units * a.lanes);
    const uint64_t ctas = (a.tokens + a.group - 1) / a.group;
    Launch l{(unsigned)std::min<uint64_t>(ctas, (uint64_t)sms * 8 * 4), kThreads, 0, stream, 0, true};
    const cudaError_t e = launch(l, k_rotary<T, N, WIDE, HALF>, a);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "rotary kernel launch");
}

template <class T, int N>
int go(Args &a, bool half, cudaStream_t stream) {
    return half ? start<T, N, true, true>(a, stream) : start<T, N, true, false>(a, stream);
}

int run(const bf16opt_rotary_t *d, const void *q, const void *k, void *out_q, void *out_k, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    auto bad = [](const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("rotary: ") + m); };
    if (!d) return bad("the descriptor is NULL");
    if (!type_ok(d->type)) return bad("unknown element type");
    if (!index_ok(d->positions_type)) return bad("unknown index type");
    if (d->layout != BF16OPT_ROTARY_HALF && d->layout != BF16OPT_ROTARY_INTERLEAVED) return bad("unknown layout");
    if (d->inverse != 0 && d->inverse != 1) return bad("inverse must be 0 or 1");
    if (d->reserved) return bad("reserved must be 0");
    if (d->heads < 1 || d->heads > (1u << 20) || d->kv_heads > (1u << 20)) return bad("heads must lie in [1, 2^20], kv_heads in [0, 2^20]");
    if (d->dim < 1 || d->dim > 65536) return bad("dim must lie in [1, 65536]");
    if (d->rotary_dim < 2 || d->rotary_dim % 2 || d->rotary_dim > d->dim || d->rotary_dim > BF16OPT_ROTARY_MAX_DIM)
        return bad("rotary_dim must be even and lie in [2, min(dim, BF16OPT_ROTARY_MAX_DIM)]");
    if (!std::isfinite(d->scale)) return bad("scale must be finite");
    if (!d->frequencies) return bad("frequencies is NULL");
    for (uint32_t i = 0; i < d->rotary_dim / 2; ++i)
        if (!std::isfinite(d->frequencies[i])) return bad("a frequency is not finite");
    if ((unsigned __int128)d->batch * d->seq >= (1ull << 40)) return bad("the sizes overflow");
    if (d->batch == 0 || d->seq == 0) return BF16OPT_OK;
    if (d->positions_stride != 0 && d->positions_stride != d->seq) return bad("positions_stride must be 0 or seq");
    if (!q || !out_q || (d->kv_heads && (!k || !out_k))) return bad("a pointer is NULL");
    Box in[2], out[2];
    const int n = d->kv_heads ? 2 : 1;
    if (!box(in[0], d, q, d->q_stride, d->heads) || !box(out[0], d, out_q, d->out_q_stride, d->heads) ||
        (n > 1 && (!box(in[1], d, k, d->k_stride, d->kv_heads) || !box(out[1], d, out_k, d->out_k_stride, d->kv_heads))))
        return bad("the sizes overflow");
    const uint64_t e = type_bytes(d->type);
    for (int i = 0; i < n; ++i)
        if (misaligned(in[i].p, e) || misaligned(out[i].p, e)) return fail(BF16OPT_ERR_ALIGNMENT, "rotary: a pointer is not aligned to its element");
    if (d->positions && misaligned(d->positions, index_bytes(d->positions_type)))
        return fail(BF16OPT_ERR_ALIGNMENT, "rotary: positions is not aligned to its element");
    const uint64_t positions = d->positions ? (d->positions_stride ? d->batch : 1) * d->seq * index_bytes(d->positions_type) : 0;
    for (int i = 0; i < n; ++i) {
        if (!apart(out[i])) return bad("an output has an element twice");
        if (overlap(out[i].p, span(out[i]), d->positions, positions)) return bad("an output overlaps an input");
        for (int j = 0; j < n; ++j)
            if (!(i == j && same(out[i], in[j])) && may_overlap(out[i], in[j])) return bad("an output overlaps an input");
    }
    if (n > 1 && may_overlap(out[0], out[1])) return bad("two outputs overlap");

    Args a = {};
    Place *place[2] = {&a.q, &a.k};
    uint64_t bits = 0;   // everything that has to be a multiple of a vector's bytes
    for (int i = 0; i < n; ++i) {
        *place[i] = Place{in[i].p, const_cast<void *>(out[i].p), in[i].s[0] / e, in[i].s[1] / e, in[i].s[2] / e, out[i].s[0] / e, out[i].s[1] / e, out[i].s[2] / e};
        bits |= (uintptr_t)in[i].p | (uintptr_t)out[i].p;
        for (int s = 0; s < 3; ++s) bits |= in[i].s[s] | out[i].s[s];
    }
    const bool half = d->layout == BF16OPT_ROTARY_HALF;
    bits |= (half ? d->rotary_dim / 2 : d->rotary_dim) * e | d->dim * e | d->rotary_dim * e;
    a.tokens = d->batch * d->seq, a.seq = d->seq;
    a.positions = d->positions, a.positions_stride = d->positions_stride, a.positions_type = d->positions_type;
    a.offset = d->offset;
    a.heads = d->heads, a.all_heads = d->heads + d->kv_heads;
    a.dim = d->dim, a.turned = d->rotary_dim;
    a.scale = d->scale, a.inverse = (uint32_t)d->inverse;
    for (uint32_t i = 0; i < d->rotary_dim / 2; ++i) {
        const double turns = d->frequencies[i] * 0.15915494309189533577;   // 1 / (2 pi)
        a.turns[i] = (uint64_t)std::llrint((turns - std::rint(turns)) * 0x1p63) << 1;   // a position is a whole number: whole turns do not count
    }
    const cudaStream_t st = (cudaStream_t)stream;
    const auto whole = [&](uint64_t n) { return bits % n == 0; };
    if (d->type == BF16OPT_TYPE_BF16) {
        if (whole(16)) return go<__nv_bfloat16, 8>(a, half, st);
        if (whole(8)) return go<__nv_bfloat16, 4>(a, half, st);
        if (whole(4)) return go<__nv_bfloat16, 2>(a, half, st);
        return half ? start<__nv_bfloat16, 1, false, true>(a, st) : start<__nv_bfloat16, 2, false, false>(a, st);
    }
    if (whole(16)) return go<float, 4>(a, half, st);
    if (whole(8)) return go<float, 2>(a, half, st);
    return half ? start<float, 1, false, true>(a, st) : start<float, 2, false, false>(a, st);
}

}  // namespace
}  // namespace bf16ops

extern "C" int bf16opt_rotary(const bf16opt_rotary_t *d, const void *q, const void *k, void *out_q, void *out_k, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::run(d, q, k, out_q, out_k, stream); });
}
