// rotary.cu -- rotary positions, forward and backward (bf16opt_rotary of include/bf16opt.h).
//
// Every element is read once and written once, which is what bounds the operator; q and k go
// in one launch.  A thread has one place in the head (a vector of elements and, in the half layout, its
// partners') and walks over tokens and heads with it; an angle's sine and cosine are computed once per token (of
// q and of k) for all the heads that it turns.
//
// The angle: position times frequency, both whole numbers (2^-64 turns), wraps around
// at whole turns by itself; what is left, in [-1/2, 1/2) turns, goes to FP32.
//
// Measured on one GB300 (a copy runs at 6.69 TB/s): 8192 tokens of 112 and 16 heads of 128 bf16, parts of one projection, 64 elements turned,
// 87 us, 6.2 TB/s; all turned (half) 91 us, 5.9 TB/s; 32 and 8 heads 35 us, 4.7 TB/s; one head of each, where every piece has sines of
// its own, 32768 tokens 27 us, 1.3 TB/s.  Sines in each thread's registers, a token's heads one batch after the other, took 109 us
// for the first, and a CTA for each group of tokens, instead of one that walks on, 49 us for the last.
#include <type_traits>

#include "ops_common.cuh"

namespace bf16ops {
namespace {

constexpr int kThreads = 256;
constexpr int kResident = 4;   // CTAs of an SM: 64 registers (pieces of four and eight bf16 spill 20 to 44 bytes)
// Heads whose pieces a thread asks for at a time: 64 bytes, at most eight pieces.
template <class T, int N, bool HALF>
constexpr int kBatchOf = std::max(1, std::min(8, 64 / (int)(N * sizeof(T))) / (HALF ? 2 : 1));

// One of q and k, and how a CTA takes it.
struct Part {
    const void *in;
    void *out;
    uint64_t in_b, in_t, in_h, out_b, out_t, out_h;   // elements between batches, tokens, heads
    uint32_t heads;
    uint32_t lanes;             // heads side by side in a CTA
    uint32_t group;             // tokens side by side in a CTA
};

struct Args {
    Part part[2];
    uint64_t tokens, seq;       // tokens: batch * seq
    const void *positions;
    uint64_t positions_stride;
    int64_t offset;
    int positions_type;
    uint32_t dim, turned;
    uint32_t units;             // threads of a head: the ones that turn, then the ones that copy
    uint32_t turning;           // of them turning
    float scale;
    uint32_t inverse;
    uint64_t turns[BF16OPT_ROTARY_MAX_DIM / 2];   // 2^-64 turns per position
};

// N elements as one access (WIDE) or as N.
template <class T, int N, bool WIDE>
struct Piece {
    T e[N];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = p[i];
    }
    __device__ __forceinline__ void store(T *p) const {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = e[i];
    }
    __device__ __forceinline__ void unpack(float (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32(e[i]);
    }
    __device__ __forceinline__ void pack(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) from_f32(e[i], f[i]);
    }
};
template <class T, int N>
struct Piece<T, N, true> {
    static constexpr int W = N * sizeof(T) / 4;
    using Word = std::conditional_t<W == 4, uint4, std::conditional_t<W == 2, uint2, unsigned int>>;
    union {
        Word v;
        uint32_t w[W];
    };
    __device__ __forceinline__ void load(const T *p) { v = __ldcs(reinterpret_cast<const Word *>(p)); }
    __device__ __forceinline__ void store(T *p) const { __stcs(reinterpret_cast<Word *>(p), v); }
    __device__ __forceinline__ void unpack(float (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 2) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
            else f[i] = __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[N]) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(T) == 2) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
            else w[i] = __float_as_uint(f[i]);
        }
    }
};

// Each product and sum spelt out, so that a result does not depend on the variant that computes it.
__device__ __forceinline__ void turned_pair(float a, float b, float c, float s, float &u, float &v) {
    u = fmaf(-b, s, __fmul_rn(a, c));
    v = fmaf(a, s, __fmul_rn(b, c));
}

__device__ __forceinline__ uint64_t position_of(const Args &a, uint64_t token) {
    const uint64_t b = a.tokens == a.seq ? 0 : token / a.seq, t = token - b * a.seq;
    return (a.positions ? (uint64_t)load_index(a.positions, a.positions_type, b * a.positions_stride + t) : t) + (uint64_t)a.offset;
}

// HALF: a thread turns N pairs (i, i + turned / 2); else N / 2 pairs of neighbours.  What is not turned is copied by threads
// of its own, in the same walk.  A CTA has `group` tokens at a time, of q and then of k: its threads ask for their pieces of
// kBatch heads, then take the tokens' sines and cosines, together, into shared memory (the positions were asked for a
// group before), and then use both.
template <class T, int N, bool WIDE, bool HALF>
__global__ void __launch_bounds__(kThreads, kResident) k_rotary(const Args a) {
    constexpr int P = HALF ? N : N / 2;       // pairs of a thread
    constexpr int V = HALF ? 2 : 1;           // pieces of a head
    constexpr int kBatch = kBatchOf<T, N, HALF>;
    constexpr uint32_t kTable = kThreads * P; // pairs of a CTA's tokens, at most
    __shared__ __align__(16) float cosines[kTable], sines[kTable];
    __shared__ uint64_t positions[kThreads];
    const uint32_t pairs = a.turned / 2, side = kThreads / pairs;   // tokens whose sines are taken side by side
    const uint32_t pair = threadIdx.x % pairs, by = threadIdx.x / pairs;
    const uint64_t turns = a.turns[pair];
    pdl_enter();
    uint64_t begun = 0;   // groups of the parts before
    for (int k = 0; k < 2; ++k) {
        const Part &pt = a.part[k];
        if (pt.heads == 0) continue;
        const uint32_t lanes = pt.lanes, group = pt.group;
        const uint64_t groups = (a.tokens + group - 1) / group;
        // the turning threads of a token first, then the copying ones: most warps do one or the other
        const uint32_t per_token = a.units * lanes, copying = a.units - a.turning;
        const uint32_t slot = threadIdx.x / per_token, left = threadIdx.x - slot * per_token;
        const bool turn = left < a.turning * lanes;
        const uint32_t rest = turn ? left : left - a.turning * lanes, each = turn ? a.turning : copying;
        const uint32_t lane = rest / each, unit = rest - lane * each;
        const uint32_t at = turn ? unit * N : a.turned + unit * N;      // the thread's first piece
        const uint32_t apart = turn ? a.turned / 2 : copying * N;       // and from it to the second
        uint32_t whole = 0;   // pieces that are there whole
#pragma unroll
        for (int v = 0; v < V; ++v) whole += turn || at + v * apart + N <= a.dim;
        const bool more = at + whole * apart < a.dim && !turn;
        const uint64_t in_step = lanes * pt.in_h, out_step = lanes * pt.out_h;
        // the groups go round the CTAs, on from where those of the part before ended
        uint64_t g = (blockIdx.x + gridDim.x - begun % gridDim.x) % gridDim.x;
        begun += groups;
        auto ask_position = [&](uint64_t g) {
            const uint64_t token = g * group + threadIdx.x;
            return threadIdx.x < group && token < a.tokens ? position_of(a, token) : 0;
        };
        uint64_t position = ask_position(g);
        for (; g < groups; g += gridDim.x) {
            const uint64_t token = g * group + slot, b = a.tokens == a.seq ? 0 : token / a.seq, t = token - b * a.seq;
            const T *in = reinterpret_cast<const T *>(pt.in) + (b * pt.in_b + t * pt.in_t + lane * pt.in_h + at);
            T *out = reinterpret_cast<T *>(pt.out) + (b * pt.out_b + t * pt.out_t + lane * pt.out_h + at);
            // this thread's heads; none where there is nothing to copy (in place)
            const uint32_t heads = slot < group && token < a.tokens && (turn || in != out) ? pt.heads : 0;
            Piece<T, N, WIDE> x[kBatch][V];
            auto ask = [&](uint32_t head) {
                const T *from = in;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (head + i * lanes < heads) {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            if (v < whole) x[i][v].load(from + v * apart);
                    }
                    from += in_step;
                }
            };
            ask(lane);
            if (threadIdx.x < group) positions[threadIdx.x] = position;
            __syncthreads();   // (the last group's sines are used, too)
            position = ask_position(g + gridDim.x);
            if (by < side)
                for (uint32_t i = by; i < group; i += side) {
                    const int32_t part = (int32_t)(positions[i] * turns >> 32);   // of a turn, in 2^-32
                    float sine, cosine;
                    sincospif((float)part * 0x1p-31f, &sine, &cosine);
                    cosines[i * pairs + pair] = cosine * a.scale;
                    sines[i * pairs + pair] = sine * (a.inverse ? -a.scale : a.scale);
                }
            __syncthreads();
            for (uint32_t head = lane; head < heads; head += lanes * kBatch) {
                float c[P], s[P];
                if (turn) {
                    const uint32_t from = slot * pairs + unit * P;
#pragma unroll
                    for (int k = 0; k < P; ++k) c[k] = cosines[from + k], s[k] = sines[from + k];
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (head + i * lanes < heads) {
                        if (turn) {
                            if constexpr (HALF) {
                                float f[N], g[N], u[N], w[N];
                                x[i][0].unpack(f), x[i][1].unpack(g);
#pragma unroll
                                for (int k = 0; k < N; ++k) turned_pair(f[k], g[k], c[k], s[k], u[k], w[k]);
                                x[i][0].pack(u), x[i][1].pack(w);
                            } else {
                                float f[N], u[N];
                                x[i][0].unpack(f);
#pragma unroll
                                for (int k = 0; k < P; ++k) turned_pair(f[2 * k], f[2 * k + 1], c[k], s[k], u[2 * k], u[2 * k + 1]);
                                x[i][0].pack(u);
                            }
                        }
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            if (v < whole) x[i][v].store(out + v * apart);
                        if (more)   // a last piece that is not whole, the rest of a long head
                            for (uint32_t k = whole * apart; at + k < a.dim; k += apart)
                                for (uint32_t e = k; e < k + N && at + e < a.dim; ++e) out[e] = in[e];
                    }
                    in += in_step, out += out_step;
                }
                if (head + lanes * kBatch < heads) ask(head + lanes * kBatch);
            }
        }
        __syncthreads();   // the next part's tables go where this one's were
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

// f radians in 2^-64 turns, to the nearest; whole turns do not count, since a position is a whole number.  The product with 1 / (2 pi)
// is a sum of two doubles: rounded to one, it is off by 2^-56 turns or so, which a position of 2^36 makes an angle's 2^-17.
uint64_t turns_of(double f) {
    constexpr double kTurn = 0.15915494309189533577, kRest = -9.839338337591243e-18;   // 1 / (2 pi), and what the double lacks of it
    double rest = 0.;   // what is left of the parts so far, less than a unit
    auto units = [&](double x) {
        x -= std::rint(x);
        const double high = x * 0x1p32, h = std::rint(high), low = (high - h) * 0x1p32 + rest, l = std::rint(low);
        rest = low - l;
        return ((uint64_t)(int64_t)h << 32) + (uint64_t)(int64_t)l;
    };
    const double p = f * kTurn;
    const uint64_t n = units(p);
    return n + units(std::fma(f, kRest, std::fma(f, kTurn, -p)));
}

template <class T, int N, bool WIDE, bool HALF>
int start(Args &a, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "rotary: no CUDA device");
    const uint32_t width = HALF ? 2 * N : N;   // elements that a thread turns
    a.turning = a.turned / width;
    // copying threads have two pieces too where the turning ones do (at most half the threads turn)
    const uint32_t pieces = (a.dim - a.turned + N - 1) / N;
    a.units = a.turning + std::min(HALF ? (pieces + 1) / 2 : pieces, (uint32_t)kThreads / 2);
    // heads side by side: a thread takes one batch of a token's heads, fewer while the SMs are not full
    constexpr uint32_t kBatch = kBatchOf<T, N, HALF>;
    uint64_t groups = 0;
    for (Part &p : a.part) {
        if (p.heads == 0) continue;
        uint32_t most = kBatch;
        while (most > 1 && a.tokens * ((p.heads + most - 1) / most) * a.units < (uint64_t)sms * 1024) most /= 2;
        p.lanes = std::min(kThreads / a.units, (p.heads + most - 1) / most);
        p.group = kThreads / (a.units * p.lanes);
        groups += (a.tokens + p.group - 1) / p.group;
    }
    Launch l{0, kThreads, 0, stream, 1, true};
    int fit = 0;   // as many as the device holds at once: each walks on
    cudaError_t e = clusters_that_fit(l, k_rotary<T, N, WIDE, HALF>, fit);
    if (e != cudaSuccess) return fail_cuda(e, "rotary occupancy");
    l.grid = (unsigned)std::min<uint64_t>(groups, fit);
    l.cluster = 0;   // (CTAs start faster without the attribute)
    e = launch(l, k_rotary<T, N, WIDE, HALF>, a);
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
    uint64_t bits = 0;   // everything that has to be a multiple of a vector's bytes
    for (int i = 0; i < n; ++i) {
        a.part[i] = Part{in[i].p, const_cast<void *>(out[i].p), in[i].s[0] / e, in[i].s[1] / e, in[i].s[2] / e,
                         out[i].s[0] / e, out[i].s[1] / e, out[i].s[2] / e, i ? d->kv_heads : d->heads, 0, 0};
        bits |= (uintptr_t)in[i].p | (uintptr_t)out[i].p;
        for (int s = 0; s < 3; ++s) bits |= in[i].s[s] | out[i].s[s];
    }
    const bool half = d->layout == BF16OPT_ROTARY_HALF;
    bits |= (half ? d->rotary_dim / 2 : d->rotary_dim) * e | d->dim * e | d->rotary_dim * e;
    a.tokens = d->batch * d->seq, a.seq = d->seq;
    a.positions = d->positions, a.positions_stride = d->positions_stride, a.positions_type = d->positions_type;
    a.offset = d->offset;
    a.dim = d->dim, a.turned = d->rotary_dim;
    a.scale = d->scale, a.inverse = (uint32_t)d->inverse;
    for (uint32_t i = 0; i < d->rotary_dim / 2; ++i) a.turns[i] = turns_of(d->frequencies[i]);
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
