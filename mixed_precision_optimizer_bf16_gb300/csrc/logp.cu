// logp.cu -- log-probabilities of given tokens, and the policy and preference losses of them, forward
// and backward (bf16opt_token_logp_*, bf16opt_policy_*, bf16opt_preference_* of include/bf16opt.h).
//
// A row leaves two numbers, its largest logit m and the sum of exp((z - m) / T); a loss gives one number
// back, its derivative c by the row's log-probability; the gradient is c / T ([j = l] - softmax_j).  So
// the forward pass reads the logits once, the backward pass reads and writes them once, and where a row's loss
// depends on that row alone (the policy loss) both go in one kernel, which has the row in registers (up to 32 KB of it), in
// shared memory (up to 72 KB) or reads it a second time while it is in L2.  A preference loss needs its sequences' sums first:
// forward, a small kernel for the pairs, backward.
//
// Measured on one GB300 (algorithmic bytes over the time; a copy of the same buffers runs at 6.69 TB/s), bf16: forward 2048 x
// 250880 150 us, 6.8 TB/s; backward 299 us, 6.9 TB/s; loss and gradient at once 353 us, 5.8 TB/s, 8192 x 32000 159 us, 6.6 TB/s,
// 8192 x 8192 48 us, 5.6 TB/s.  The one-pass kernel of long rows is bound by what happens between its passes: CTAs of a cluster
// wait for one another (issue 55 %, 67 % of the warps active), and a row per CTA would not stay in L2.  What was tried for them
// instead: rows in registers across a cluster (16 vectors a thread, two CTAs of an SM: 442 us), in shared memory across a
// cluster (360 us), a CTA of 1024 threads per SM with a ring (436 us, issue 81 %).
#include <cooperative_groups.h>

#include <type_traits>

#include "logits.cuh"

namespace cg = cooperative_groups;

namespace bf16ops {
namespace {

constexpr int kThreads = 256, kFew = 64, kSome = 128, kMany = 384;   // of a CTA; for short rows; where a slice stays in shared memory
constexpr int kU = 4;              // vectors of a thread at a time
constexpr int kMaxCluster = 8;
constexpr int kPairThreads = 512;
constexpr uint64_t kSliceVectors = 2 * kThreads * kU;   // of the backward kernel's CTAs (twice as many: 1021 x 32003 FP32 55 us, 48 so; half: 2048 x 250880 341 us, 298)
// A row whose largest logit m is below this (|m| / T, in powers of two) has its exponents z c - m c in one
// instruction for two logits: the product is exact, and m c is off by its rounding (2^-4 at most), the same for the
// whole row, which goes into the row's factor.  Beyond, they are formed from the differences z - m, with m known.
constexpr float kFar = 0x1p20f;

// Of rows that are read a second time, at a time: what L2 keeps of them (two dies, each of which holds what its SMs ask
// for: at 95 MB 2048 x 250880 took 419 us instead of 341, at 76 MB 1024 x 250880 FP32 405 us, 426 us at 57; other lengths were not
// timed with other limits).
constexpr uint64_t kInFlight = 76 << 20;
constexpr unsigned kResident = 6;   // CTAs of an SM there (five: 350 us)
constexpr uint64_t kStage = 72 * 1024 / 16;   // vectors of a slice in shared memory

enum Kind { LOGP, POLICY, PREFER };

struct Args {
    uint64_t rows;
    uint32_t vocab, slices;
    const void *logits;
    uint64_t logits_stride;
    const void *labels;
    int labels_type;
    const float *row_weight;
    float c;                       // log2(e) / T
    float inv_t, inv_t_rest;       // 1 / T, and what it lacks
    // policy
    const float *advantage, *old_logp, *ref_logp;
    float lowest, highest, kl_weight;   // of the ratio
    // preference
    const void *offsets;
    int offsets_type;
    uint64_t pairs;

    const float4 *saved_in;
    const float *dloss;
    uint64_t losses;
    float *loss, *logp;
    float4 *saved;
    void *dlogits;
    uint64_t dlogits_stride;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// A stream's largest number and the sum of exp2((z - m) c).
struct Stat {
    float m, s;
};
__device__ __forceinline__ Stat warp_join(const Stat &a, float c) {
    Stat r;
    r.m = warp_max(a.m);
    r.s = warp_sum(a.s * ex2((a.m - safe_max(r.m)) * c));
    return r;
}
// (A sum that is not finite belongs to a row that is NaN, or far and summed once more.)

template <bool FAR>
__device__ __forceinline__ float2 exponent(float2 z, float m, float mc, float c) {
    if (FAR) return mul2(add2(z, both(-m)), both(c));
    return fma2(z, both(c), both(-mc));
}

// One thread's vectors of a slice, kThreads apart: groups of U of them, the first of which it asks for before anything else.  HELD: the
// slice is no longer than that and stays in registers.
template <class T, int kThreads, int U>
struct Group {
    uint4 q[U];
    __device__ __forceinline__ void load(const uint4 *zv, uint32_t i, uint32_t nv) {
        if (i + (U - 1) * kThreads < nv) {
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = zv[i + u * kThreads];
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = i + u * kThreads < nv ? zv[i + u * kThreads] : nothing<T>();
        }
    }
};

// A thread's maximum and sum so far.  FAR: around the row's largest logit, which is known.
template <class T, bool FAR>
struct Running {
    float m, mc;
    float2 sum;
    __device__ __forceinline__ explicit Running(float top) : m(FAR ? top : -INFINITY), mc(0.f), sum(both(0.f)) {}
    template <int U>
    __device__ __forceinline__ void add(const uint4 (&q)[U], float c) {
        constexpr int P = Vec<T>::N / 2;
        if (!FAR) {
            const float mx = largest<T, U>(q);
            if (mx > m) {
                const float to = fmaxf(fminf(mx * c, kFar), -kFar);
                sum = mul2(sum, both(m == -INFINITY ? 0.f : ex2(mc - to)));
                m = mx, mc = to;
            }
        }
        // each vector's terms by themselves first: beside a tall token's term, tiny ones are lost one by one (the sums of 3081 x 250880
        // bf16 were 2e-7 too small, all of them, which a sequence adds up: its loss was 8e-7 to 1.4e-6 off, 6e-8 to 2e-7 so)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[P], part = both(0.f);
            pairs<T>(q[u], f);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const float2 d = exponent<FAR>(f[k], safe_max(m), mc, c);
                const float2 e = make_float2(ex2(d.x), ex2(d.y));
                part = k ? add2(part, e) : e;
            }
            sum = add2(sum, part);
        }
    }
    // with the element at a row's end that is this thread's, if any
    __device__ __forceinline__ Stat result(float c, bool one, float f) {
        Stat st = {m, sum.x + sum.y};
        // mc is m c rounded, or -kFar: what is lost there is 2^-126 of a row that is not far
        if (!FAR && st.s != 0.f) st.s *= ex2(fmaf(-m, c, mc));
        if (one) {
            const float top = FAR ? m : fmaxf(m, f);   // (a NaN passed over)
            const float b = safe_max(top);
            st.s = st.s * ex2((m - b) * c) + ex2((f - b) * c);
            st.m = top;
        }
        return st;
    }
};

// a + b, and what rounding took off it (Knuth).
__device__ __forceinline__ float two_sum(float a, float b, float &off) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    off = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    return s;
}

// What a row's loss needs beside its logits, asked for with the first of them.
struct Given {
    float w, advantage, old_logp, ref_logp, dloss;
};
template <int KIND, bool GRAD>
__device__ __forceinline__ Given given_of(const Args &a, uint64_t row) {
    Given g = {1.f, 0.f, 0.f, 0.f, 1.f};
    if (a.row_weight) g.w = a.row_weight[row];
    if (KIND == POLICY) {
        g.advantage = a.advantage[row];
        if (a.old_logp) g.old_logp = a.old_logp[row];
        if (a.ref_logp) g.ref_logp = a.ref_logp[row];
    }
    if (GRAD && a.dloss) g.dloss = a.dloss[row];
    return g;
}

// A number as a sum of two, hi the nearest to it; lo 0 beside an infinite or NaN hi.  A sum is off by 2^-47 of it at most where both have the
// same sign (what rounding takes off the two small additions), and hi and lo are made apart again each time: small terms would else
// gather in lo, which alone is an FP32 sum.
struct Two {
    float hi, lo;
    __device__ __forceinline__ Two operator+(const Two &b) const {   // (a + b and b + a are the same bits)
        float off, rest;
        const float s = two_sum(hi, b.hi, off), h = two_sum(s, __fadd_rn(__fadd_rn(lo, b.lo), off), rest);
        return fabsf(h) < INFINITY ? Two{h, rest} : Two{s, 0.f};
    }
    __device__ __forceinline__ float value() const { return hi + lo; }
};

// A row's log-probability (z - m) / T - log s.  log s = k ln 2 + log f, f in [0.7, 1.4], ln 2 as its leading bits, k times which is
// exact, and the rest (Cody and Waite's reduction).
__device__ __forceinline__ Two logp_of(const Args &a, float m, float s, float z) {
    float off;
    const float d = two_sum(z, -m, off), p = d * a.inv_t;
    if (!(fabsf(p) < INFINITY && s > 0.f && s < INFINITY)) {
        if (m == -INFINITY && s == 0.f) return {-INFINITY, 0.f};
        // (a difference that no FP32 number holds, of numbers of opposite signs, may be one when it is divided)
        return {(fabsf(d) < INFINITY ? p : z * a.inv_t - m * a.inv_t) - logf(s), 0.f};
    }
    int k;
    float f = frexpf(s, &k);
    if (f < 0.70710678f) f *= 2.f, --k;
    constexpr float kLn2 = 0.693145751953125f, kLn2Rest = (float)(0.69314718055994530942 - (double)kLn2);
    const float lo = fmaf(d, a.inv_t, -p) + fmaf(d, a.inv_t_rest, off * a.inv_t) - fmaf((float)k, kLn2Rest, logf(f));
    return Two{p, lo} + Two{-kLn2 * (float)k, 0.f};
}

// A counted row's log-probability, loss and slope.  The log-probability stays a sum of two numbers until it is compared with the others', so
// that a ratio is as exact as its exponential.
struct Terms {
    float loss, logp, slope;
};
template <int KIND>
__device__ __forceinline__ Terms terms_of(const Args &a, const Given &g, float m, float s, float z) {
    Terms t;
    const Two logp = logp_of(a, m, s, z);
    t.logp = logp.value();
    t.loss = 0.f, t.slope = 1.f;
    if (KIND == POLICY) {
        // of its own tokens the ratio is the constant 1, an infinite log-probability's too; NaN stays
        const float x = a.old_logp ? (logp + Two{-g.old_logp, 0.f}).value() : t.logp == t.logp ? 0.f : t.logp;
        const float adv = g.advantage, ratio = expf(x);
        const float kept = adv >= 0.f ? (ratio > a.highest ? a.highest : ratio) : (ratio < a.lowest ? a.lowest : ratio);   // NaN stays
        t.loss = -kept * adv;
        t.slope = kept == ratio || ratio != ratio ? -ratio * adv : 0.f;
        if (a.ref_logp) {
            const float d = (Two{g.ref_logp, 0.f} + Two{-logp.hi, -logp.lo}).value(), e = expm1f(d);
            t.loss += a.kl_weight * (d == INFINITY ? d : e - d);
            t.slope -= a.kl_weight * e;
        }
        t.loss *= g.w, t.slope *= g.w;
    }
    return t;
}

// A slice of a row's gradient: vectors [v0, v0 + nv), with the elements before the first or behind the last vector of the row.
template <class T>
struct Target {
    const T *z;
    T *out;
    uint32_t head, v0, nv, tail0, vocab;
    bool first, last;   // the slice has the row's ends
    __device__ __forceinline__ bool whole() const { return (((uintptr_t)out ^ (uintptr_t)z) & 15u) == 0; }
    __device__ __forceinline__ T *vectors() const { return out + head + (size_t)v0 * Vec<T>::N; }
};

// scale_q exp2((z - m) c), and scale at the label.
template <class T, bool FAR, int kThreads>
struct Gradient {
    static constexpr int N = Vec<T>::N, P = N / 2;
    float base, mc, c, factor, scale;
    uint32_t label, own, lane;   // own: the vector of the slice that has the label, if it is this thread's; the label's place in it
    T *ov;
    bool whole;
    __device__ __forceinline__ Gradient(const Target<T> &t, float m, float c_, float scale_q, float scale_, uint32_t label_)
        : base(safe_max(m)), mc(base * c_), c(c_), factor(FAR ? scale_q : scale_q * ex2(fmaf(-base, c_, mc))), scale(scale_), label(label_), ov(t.vectors()),
          whole(t.whole()) {
        const uint32_t at = label - t.head - t.v0 * N;
        own = label >= t.head && at / N < t.nv && at / N % kThreads == threadIdx.x ? at / N : 0xffffffffu;
        lane = at % N;
    }
    __device__ __forceinline__ void put(const uint4 &q, uint32_t j) const {
        float2 f[P];
        pairs<T>(q, f);
        float g[N];
#pragma unroll
        for (int k = 0; k < P; ++k) {
            const float2 d = exponent<FAR>(f[k], base, mc, c);
            const float2 r = mul2(both(factor), make_float2(ex2(d.x), ex2(d.y)));
            g[2 * k] = r.x, g[2 * k + 1] = r.y;
        }
        if (j == own) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (lane == k) g[k] += scale;
        }
        store_vec<T>(ov + (size_t)j * N, g, whole);
    }
    __device__ __forceinline__ void ends(const Target<T> &t) const {
        auto one = [&](uint32_t at) {
            const float f = to_f32(t.z[at]);
            const float2 d = exponent<FAR>(make_float2(f, f), base, mc, c);
            from_f32(t.out[at], fmaf(factor, ex2(d.x), at == label ? scale : 0.f));
        };
        if (t.first && threadIdx.x < t.head) one(threadIdx.x);
        if (t.last && threadIdx.x < t.vocab - t.tail0) one(t.tail0 + threadIdx.x);
    }
};

template <class T, bool FAR, int kThreads>
__device__ __forceinline__ void grad_slice(const Target<T> &t, float m, float c, float scale_q, float scale, uint32_t label) {
    const Gradient<T, FAR, kThreads> g(t, m, c, scale_q, scale, label);
    const uint4 *zv = reinterpret_cast<const uint4 *>(t.z + t.head) + t.v0;
    for (uint32_t i = threadIdx.x; i < t.nv; i += kThreads * kU) {
        uint4 q[kU];
        if (i + (kU - 1) * kThreads < t.nv) {
#pragma unroll
            for (int u = 0; u < kU; ++u) q[u] = zv[i + u * kThreads];
#pragma unroll
            for (int u = 0; u < kU; ++u) g.put(q[u], i + u * kThreads);
        } else {
            for (uint32_t j = i; j < t.nv; j += kThreads) g.put(zv[j], j);
        }
    }
    g.ends(t);
}

template <class T, int kThreads>
__device__ __forceinline__ void zero_slice(const Target<T> &t) {
    constexpr int N = Vec<T>::N;
    T *ov = t.vectors();
    const bool whole = t.whole();
    const float zero[N] = {};
    for (uint32_t i = threadIdx.x; i < t.nv; i += kThreads) store_vec<T>(ov + (size_t)i * N, zero, whole);
    if (t.first && threadIdx.x < t.head) from_f32(t.out[threadIdx.x], 0.f);
    if (t.last && threadIdx.x < t.vocab - t.tail0) from_f32(t.out[t.tail0 + threadIdx.x], 0.f);
}

__device__ __forceinline__ bool far_row(float m, float c) { return !(fabsf(m * c) < kFar) && m != -INFINITY; }

constexpr int kStaged = -1;

// A cluster of CTAs (or one) takes a row.  HELD vectors of a thread stay in registers between the two passes: the slice is
// no longer than that.  kStaged: it comes through, and stays in, shared memory, where each thread has places of its own.  0: it is
// read again.
template <class T, int KIND, bool GRAD, int kThreads, int HELD>
__global__ void __launch_bounds__(kThreads, HELD == 8 || HELD == kStaged ? (kThreads == kSome ? 6 : 3) : kThreads == kFew ? 16 : kThreads == kSome ? 8
                                                        : GRAD && HELD == 0 ? kResident : 5) k_rows(const Args a) {
    constexpr bool STAGED = HELD == kStaged;
    constexpr int U = HELD > 0 ? HELD : kU, kWarps = kThreads / 32;
    extern __shared__ __align__(128) uint4 stage[];
    __shared__ Stat sm[2][kMaxCluster * kWarps];
    __shared__ float sm_scale;
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint64_t row = blockIdx.x / ranks;
    if (ranks > 1) cluster_arrive();   // (every CTA's shared memory has to exist before another one writes there)
    pdl_enter();
    const T *z = reinterpret_cast<const T *>(a.logits) + row * a.logits_stride;
    const Slice s = slice_of(z, a.vocab, rank, ranks, 31 - __clz(ranks));
    const uint4 *zv = reinterpret_cast<const uint4 *>(z + s.head) + s.v0;
    const uint32_t nv = s.v1 - s.v0;
    // asked for before it is known whether the row counts: of one that does not, all that is held (up to 72 KB), else the first group, is read
    Group<T, kThreads, U> group;
    uint32_t groups = 0;   // of copies on their way
    if constexpr (STAGED) {
        for (uint32_t i = tid; i < nv + tid; i += kThreads * U, ++groups) {   // (the same number of turns for all)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * kThreads < nv) copy_async16(stage + i + u * kThreads, zv + i + u * kThreads);
            copy_commit();
        }
    } else {
        group.load(zv, tid, nv);
    }
    const int64_t label = load_index(a.labels, a.labels_type, row);
    const Given given = given_of<KIND, GRAD>(a, row);
    float w = given.w;
    if (KIND == PREFER && a.pairs == 0) {
        w = 0.f;
    } else if (KIND == PREFER) {
        const int64_t lo = load_index(a.offsets, a.offsets_type, 0), hi = load_index(a.offsets, a.offsets_type, 2 * a.pairs);
        if ((int64_t)row < lo || (int64_t)row >= hi) w = 0.f;
    }
    const bool counts = w != 0.f && label >= 0 && label < (int64_t)a.vocab;
    const Target<T> target = {z, GRAD ? reinterpret_cast<T *>(a.dlogits) + row * a.dlogits_stride : nullptr, s.head, s.v0, nv, s.tail0, a.vocab,
                              rank == 0, rank + 1 == ranks};
    if (ranks > 1) cluster_wait();
    if (!counts) {   // the same in the whole cluster
        if constexpr (STAGED) copy_wait<0>();
        if (GRAD) zero_slice<T, kThreads>(target);
        if (rank == 0 && tid == 0) {
            if (KIND == POLICY) a.loss[row] = 0.f;
            if (KIND != PREFER && a.logp) a.logp[row] = 0.f;
            if (!GRAD && a.saved) a.saved[row] = make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
        }
        pdl_leave();
        return;
    }
    const float z_label = to_f32(z[label]);
    uint32_t at = 0xffffffffu;
    if (target.first && tid < s.head) at = tid;
    else if (target.last && tid >= 32 && tid - 32 < a.vocab - s.tail0) at = s.tail0 + tid - 32;
    const float z_end = at != 0xffffffffu ? to_f32(z[at]) : 0.f;

    auto joined = [&](Stat st, int turn) {
        st = warp_join(st, a.c);
        if (lane < ranks) {
            Stat *to = &sm[turn][rank * kWarps + warp];
            *(ranks > 1 ? cluster.map_shared_rank(to, lane) : to) = st;
        }
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        Stat all = lane < ranks * kWarps ? sm[turn][lane] : Stat{-INFINITY, 0.f};
        for (uint32_t i = lane + 32; i < ranks * kWarps; i += 32) {
            const Stat b = sm[turn][i];
            const float m = fmaxf(all.m, b.m), t = safe_max(m);
            all.s = all.s * ex2((all.m - t) * a.c) + b.s * ex2((b.m - t) * a.c);
            all.m = m;
        }
        return warp_join(all, a.c);
    };
    uint32_t last = tid;   // where the group that is in registers begins
    auto pass = [&](auto far, float top) {
        Running<T, decltype(far)::value> run(top);
        if constexpr (STAGED) {
            for (uint32_t i = tid, left = groups; i < nv + tid; i += kThreads * U) {
                copy_wait_for(--left);
                group.load(stage, i, nv);
                run.add(group.q, a.c);
            }
        } else if constexpr (HELD > 0) {
            run.add(group.q, a.c);
        } else {
            if (decltype(far)::value) group.load(zv, tid, nv);
            for (last = tid;; last += kThreads * U) {
                run.add(group.q, a.c);
                if (last + kThreads * U >= nv) break;
                group.load(zv, last + kThreads * U, nv);
            }
        }
        return run.result(a.c, at != 0xffffffffu, z_end);
    };
    Stat st = joined(pass(std::false_type(), 0.f), 0);
    const bool far = far_row(st.m, a.c);
    if (far) st = joined(pass(std::true_type(), st.m), 1);

    if (!GRAD && (rank != 0 || tid != 0)) return;
    float4 keep = make_float4(st.m, st.s, 0.f, __int_as_float((int)row));
    float scale = 0.f;
    if (KIND != PREFER && warp == 0) {
        const Terms t = terms_of<KIND>(a, given, st.m, st.s, z_label);
        if (rank == 0 && tid == 0) {
            if (KIND == POLICY) a.loss[row] = t.loss;
            if (a.logp) a.logp[row] = t.logp;
        }
        keep.z = t.slope;
        if (GRAD && tid == 0) sm_scale = t.slope * given.dloss * a.inv_t;
    }
    if (!GRAD) {
        if (a.saved) a.saved[row] = keep;
        return;
    }
    __syncthreads();
    scale = sm_scale;
    auto gradient = [&](auto far) {
        constexpr bool FAR = decltype(far)::value;
        const float scale_q = st.s == 0.f ? 0.f : -scale / st.s;
        if constexpr (STAGED) {
            const Gradient<T, FAR, kThreads> g(target, st.m, a.c, scale_q, scale, (uint32_t)label);
#pragma unroll 4
            for (uint32_t j = tid; j < nv; j += kThreads) g.put(stage[j], j);
            g.ends(target);
        } else if constexpr (HELD > 0) {
            const Gradient<T, FAR, kThreads> g(target, st.m, a.c, scale_q, scale, (uint32_t)label);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (tid + u * kThreads < nv) g.put(group.q[u], tid + u * kThreads);
            g.ends(target);
        } else {
            // backwards, what was read last first: the last group is in registers, the ones before it are the likeliest to be in L2
            const Gradient<T, FAR, kThreads> g(target, st.m, a.c, scale_q, scale, (uint32_t)label);
            for (uint32_t i = last;; i -= kThreads * U) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u * kThreads < nv) g.put(group.q[u], i + u * kThreads);
                if (i < kThreads * U) break;
                group.load(zv, i - kThreads * U, nv);
            }
            g.ends(target);
        }
    };
    if (scale == 0.f) zero_slice<T, kThreads>(target);
    else if (far) gradient(std::true_type());
    else gradient(std::false_type());
    pdl_leave();
}

// The backward pass: a CTA takes a slice of a row.
template <class T>
__global__ void __launch_bounds__(kThreads) k_backward(const Args a) {
    pdl_enter();
    const uint64_t row = blockIdx.x / a.slices;
    const uint32_t slice = (uint32_t)(blockIdx.x - row * a.slices);
    const float4 keep = a.saved_in[row];
    const int index = __float_as_int(keep.w);
    float scale = 0.f;
    if (index >= 0 && (!a.dloss || (uint64_t)index < a.losses)) scale = keep.z * (a.dloss ? a.dloss[index] : 1.f) * a.inv_t;
    const T *z = reinterpret_cast<const T *>(a.logits) + row * a.logits_stride;
    const Slice s = slice_of(z, a.vocab, 0, 1, 0);
    const uint32_t v0 = (uint32_t)((uint64_t)s.nv * slice / a.slices), nv = (uint32_t)((uint64_t)s.nv * (slice + 1) / a.slices) - v0;
    const Target<T> target = {z, reinterpret_cast<T *>(a.dlogits) + row * a.dlogits_stride, s.head, v0, nv, s.tail0, a.vocab,
                              slice == 0, slice + 1 == a.slices};
    if (scale == 0.f) {
        zero_slice<T, kThreads>(target);
    } else {
        const int64_t label = load_index(a.labels, a.labels_type, row);
        const uint32_t at = label >= 0 && label < (int64_t)a.vocab ? (uint32_t)label : 0xffffffffu;
        const float scale_q = keep.y == 0.f ? 0.f : -scale / keep.y;
        if (far_row(keep.x, a.c)) grad_slice<T, true, kThreads>(target, keep.x, a.c, scale_q, scale, at);
        else grad_slice<T, false, kThreads>(target, keep.x, a.c, scale_q, scale, at);
    }
    pdl_leave();
}

// ------------------------------------------------------------------ pairs of sequences

struct PairArgs {
    Args a;
    int kind, mean;
    float beta, smoothing, margin;
    double centre;   // 1 / (2 beta)
    const float *ref;
};

// A CTA takes a pair: its sums, its loss, and its rows' slopes.  The two sequences are one range of rows, so that the loads that wait
// for one another (offsets, saved numbers and labels, the labels' logits) are waited for once; sums are pairs of FP32 numbers,
// and what is computed in 64 bits is one warp's (with sums in 64 bits, one sequence after the other: 14 us for 24 or 300 rows).
template <class T>
__global__ void __launch_bounds__(kPairThreads) k_pairs(const PairArgs p) {
    constexpr int kWarps = kPairThreads / 32;
    __shared__ int sm_offset[2][kWarps], sm_count[2][kWarps];
    __shared__ Two sm_sum[2][kWarps];
    __shared__ float sm_slope[2];
    const Args &a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_enter();
    const uint32_t n = 2 * (uint32_t)a.pairs, first = blockIdx.x, second = blockIdx.x + (uint32_t)a.pairs;
    auto offset = [&](uint32_t i) {   // within the rows
        const int64_t o = load_index(a.offsets, a.offsets_type, i);
        return (int)(o < 0 ? 0 : o > (int64_t)a.rows ? (int64_t)a.rows : o);
    };
    // the offsets that count: the largest so far, at most the last one
    const int end = offset(n), behind[2] = {offset(first + 1), offset(second + 1)};
    int most[2] = {0, 0};
    for (uint32_t j = tid; j <= second; j += kPairThreads) {
        const int o = offset(j);
        most[1] = max(most[1], o);
        if (j <= first) most[0] = max(most[0], o);
    }
    for (int k = 0; k < 2; ++k) {
        most[k] = __reduce_max_sync(0xffffffffu, most[k]);
        if (lane == 0) sm_offset[k][warp] = most[k];
    }
    __syncthreads();
    int lo[2], len[2];
    for (int k = 0; k < 2; ++k) {
        lo[k] = min(end, __reduce_max_sync(0xffffffffu, sm_offset[k][lane % kWarps]));
        len[k] = max(0, min(end, behind[k]) - lo[k]);
    }
    const uint32_t all = (uint32_t)len[0] + (uint32_t)len[1];   // below 2^32
    auto row_of = [&](uint32_t t) { return t < (uint32_t)len[0] ? (uint64_t)lo[0] + t : (uint64_t)lo[1] + (t - (uint32_t)len[0]); };
    Two sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
    int count[2] = {0, 0};
    for (uint64_t t = tid; t < all; t += kPairThreads) {
        const uint64_t r = row_of((uint32_t)t);
        const float4 keep = a.saved[r];
        const int64_t label = load_index(a.labels, a.labels_type, r);
        if (__float_as_int(keep.w) < 0) continue;
        const Two logp = logp_of(a, keep.x, keep.y, to_f32(reinterpret_cast<const T *>(a.logits)[r * a.logits_stride + label]));
        const bool k = t >= (uint32_t)len[0];
        if (k) sum[1] = sum[1] + logp, ++count[1];
        else sum[0] = sum[0] + logp, ++count[0];
    }
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum[k] = sum[k] + Two{__shfl_xor_sync(0xffffffffu, sum[k].hi, o), __shfl_xor_sync(0xffffffffu, sum[k].lo, o)};
        count[k] = __reduce_add_sync(0xffffffffu, count[k]);
        if (lane == 0) sm_sum[k][warp] = sum[k], sm_count[k][warp] = count[k];
    }
    __syncthreads();
    if (warp == 0) {
        double total[2];
        for (int k = 0; k < 2; ++k) {
            sum[k] = sm_sum[k][lane % kWarps];
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1)
                sum[k] = sum[k] + Two{__shfl_xor_sync(0xffffffffu, sum[k].hi, o), __shfl_xor_sync(0xffffffffu, sum[k].lo, o)};
            count[k] = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm_count[k][lane] : 0);
            total[k] = (double)sum[k].hi + sum[k].lo;
            if (p.mean && count[k] > 0) total[k] /= (double)count[k];
        }
        double h = total[0] - total[1];
        if (p.ref) h = (total[0] - p.ref[first]) - (total[1] - p.ref[second]);
        float loss, slope;   // slope: by h
        if (p.kind == BF16OPT_PREFER_IPO) {
            const double d = h - p.margin - p.centre;
            loss = (float)(d * d), slope = 2.f * (float)d;
        } else {
            const float m = (float)(h * p.beta - p.margin);
            if (p.kind == BF16OPT_PREFER_HINGE) {
                loss = m < 1.f ? 1.f - m : m == m ? 0.f : m;
                slope = m < 1.f ? -p.beta : m == m ? 0.f : m;
            } else {
                const float e = expf(-fabsf(m)), soft = log1pf(e);
                const float up = m >= 0.f ? 1.f / (1.f + e) : e / (1.f + e), down = m >= 0.f ? e / (1.f + e) : 1.f / (1.f + e);   // sigmoid(m), sigmoid(-m)
                const float q = p.smoothing;
                loss = (1.f - q) * (soft + (m < 0.f ? -m : 0.f)) + (q != 0.f ? q * (soft + (m > 0.f ? m : 0.f)) : 0.f);
                slope = p.beta * (q * up - (1.f - q) * down);
            }
        }
        if (lane == 0) {
            a.loss[first] = loss;
            a.logp[first] = (float)total[0], a.logp[second] = (float)total[1];
            for (int k = 0; k < 2; ++k) sm_slope[k] = (k ? -slope : slope) * (p.mean && count[k] > 0 ? 1.f / (float)count[k] : 1.f);
        }
    }
    __syncthreads();
    for (uint64_t t = tid; t < all; t += kPairThreads) {
        float4 &keep = a.saved[row_of((uint32_t)t)];
        if (__float_as_int(keep.w) >= 0) keep.z = sm_slope[t >= (uint32_t)len[0]], keep.w = __int_as_float((int)blockIdx.x);
    }
    pdl_leave();
}

// ---------------------------------------------------------------------- host

struct Part {
    const void *p;
    uint64_t n;
};

int bad(const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("logp: ") + m); }

// What the calls share: the descriptor, then the outputs against the inputs and one another.  `in` and `outs`: 4-byte
// aligned arrays; `grad`: dlogits is written.
int check(const bf16opt_tokens_t *d, std::initializer_list<Part> in, std::initializer_list<Part> outs, const void *dlogits,
          uint64_t dlogits_stride, bool grad) {
    const uint64_t eb = type_bytes(d->logits_type);
    uint64_t zb = 0, gb = 0;
    if (d->logits_stride < d->vocab || (grad && dlogits_stride < d->vocab)) return bad("a row stride is below vocab");
    if (!span_bytes(d->rows, d->logits_stride, d->vocab, eb, zb) || (grad && !span_bytes(d->rows, dlogits_stride, d->vocab, eb, gb)))
        return bad("the sizes overflow");
    const auto unaligned = [] { return fail(BF16OPT_ERR_ALIGNMENT, "logp: a pointer is not aligned to its element"); };
    if (d->rows) {   // (of no rows there are still a preference's losses, sums and offsets)
        if (!d->logits || !d->labels) return bad("an input pointer is NULL");
        if (grad && !dlogits) return bad("dlogits is NULL");
        if (misaligned(d->logits, eb) || misaligned(dlogits, eb) || misaligned(d->labels, index_bytes(d->labels_type)) || misaligned(d->row_weight, 4))
            return unaligned();
        for (auto *parts : {&in, &outs})
            for (const Part &x : *parts)
                if (misaligned(x.p, 4)) return unaligned();
    }
    const Part own[] = {{d->logits, zb}, {d->labels, d->rows * index_bytes(d->labels_type)}, {d->row_weight, d->rows * 4}};
    const Part dz = {grad ? dlogits : nullptr, gb};
    auto meets = [&](const Part &o, bool gradient) {
        for (const Part &x : own) {
            if (gradient && x.p == d->logits && dlogits == d->logits && dlogits_stride == d->logits_stride) continue;   // in place
            if (overlap(o.p, o.n, x.p, x.n)) return true;
        }
        for (const Part &x : in)
            if (overlap(o.p, o.n, x.p, x.n)) return true;
        return false;
    };
    if (meets(dz, true)) return bad("an output overlaps an input");
    for (const Part *o = outs.begin(); o != outs.end(); ++o) {
        if (meets(*o, false)) return bad("an output overlaps an input");
        if (overlap(o->p, o->n, dz.p, dz.n)) return bad("two outputs overlap");
        for (const Part *q = outs.begin(); q != o; ++q)
            if (overlap(o->p, o->n, q->p, q->n)) return bad("two outputs overlap");
    }
    return BF16OPT_OK;
}

int check_tokens(const bf16opt_tokens_t *d) {
    if (!d) return bad("the descriptor is NULL");
    if (!type_ok(d->logits_type)) return bad("unknown element type");
    if (!index_ok(d->labels_type)) return bad("unknown index type");
    if (d->vocab < 1 || d->vocab > (1u << 30)) return bad("vocab must lie in [1, 2^30]");
    if (d->rows > BF16OPT_TOKENS_MAX_ROWS) return bad("rows exceeds BF16OPT_TOKENS_MAX_ROWS");
    if (!(std::isfinite(d->temperature) && d->temperature > 0.f) || !std::isfinite(1.f / d->temperature) ||
        !((float)(1.4426950408889634074 / (double)d->temperature) < 1e36f))
        return bad("temperature must be finite and > 0, with a finite reciprocal");
    return BF16OPT_OK;
}

Args args_of(const bf16opt_tokens_t *d) {
    Args a = {};
    a.rows = d->rows, a.vocab = d->vocab;
    a.logits = d->logits, a.logits_stride = d->logits_stride;
    a.labels = d->labels, a.labels_type = d->labels_type, a.row_weight = d->row_weight;
    const double inv_t = 1.0 / (double)d->temperature;
    a.inv_t = (float)inv_t, a.inv_t_rest = (float)(inv_t - (double)a.inv_t);
    a.c = (float)(1.4426950408889634074 / (double)d->temperature);
    return a;
}

template <class T, int KIND, bool GRAD, int kThreads, int HELD>
int launch_rows(const Args &a, unsigned cluster, cudaStream_t stream, size_t smem = 0) {
    auto k = k_rows<T, KIND, GRAD, kThreads, HELD>;
    // (CTAs start faster without the attribute: 8192 x 1268 both ways 19 us, 27 us as clusters of one)
    const Launch l{(unsigned)(a.rows * cluster), (unsigned)kThreads, smem, stream, cluster > 1 || smem ? cluster : 0, true};
    if (smem) {
        int fit = 0;   // (allows the kernel its shared memory)
        const cudaError_t e = clusters_that_fit(l, k, fit);
        if (e != cudaSuccess) return fail_cuda(e, "logp occupancy");
    }
    const cudaError_t e = launch(l, k, a);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "logp kernel launch");
}

template <class T, int KIND, bool GRAD>
int choose_rows(const Args &a, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "logp: no CUDA device");
    const uint64_t vecs = a.vocab / Vec<T>::N;   // of a row, at most
    // CTAs per row: as many as keep the SMs busy with few rows
    unsigned cluster = 1;
    while (cluster < kMaxCluster && a.rows * cluster <= (uint64_t)sms * 4 && vecs / cluster > 2 * kThreads * kU) cluster *= 2;
    // fewer threads for short rows, so that each has several vectors on their way (8192 x 3000 both ways 31 us, 45 us with 256 threads)
    if (vecs <= kFew * kU) return launch_rows<T, KIND, GRAD, kFew, GRAD ? kU : 0>(a, 1, stream);
    if (cluster == 1 && vecs <= kSome * kU) return launch_rows<T, KIND, GRAD, kSome, GRAD ? kU : 0>(a, 1, stream);
    if (cluster == 1 && vecs <= kSome * 8) return launch_rows<T, KIND, GRAD, kSome, GRAD ? 8 : 0>(a, 1, stream);
    if constexpr (GRAD) {
        // in registers; or in shared memory, where a CTA's part of it is enough (several CTAs per row wait for one another: 2048 x 128256
        // took 184 us either way, 4096 x 50257 170 us, 145 us from L2)
        if (vecs <= (uint64_t)cluster * kThreads * 4) return launch_rows<T, KIND, GRAD, kThreads, 4>(a, cluster, stream);
        if (vecs <= (uint64_t)cluster * kThreads * 8) return launch_rows<T, KIND, GRAD, kThreads, 8>(a, cluster, stream);
        if (cluster == 1 && vecs <= kStage) return launch_rows<T, KIND, GRAD, kMany, kStaged>(a, 1, stream, vecs * 16);
        // the second pass from L2: so many CTAs per row, and so few of an SM, that what the SMs have of rows at a time stays there
        const uint64_t row = vecs * 16, all = a.rows * row;
        while (cluster < kMaxCluster && sms * kResident / cluster * row > kInFlight && all > kInFlight) cluster *= 2;
        const uint64_t resident = std::max<uint64_t>(2, kInFlight * cluster / (sms * row));
        const bool fewer = resident < kResident && all > kInFlight;
        return launch_rows<T, KIND, GRAD, kThreads, 0>(a, cluster, stream, fewer ? 224 * 1024 / (resident + 1) : 0);
    }
    return launch_rows<T, KIND, GRAD, kThreads, 0>(a, cluster, stream);
}

template <int KIND, bool GRAD>
int rows_kernel(const Args &a, int type, void *stream) {
    return type == BF16OPT_TYPE_BF16 ? choose_rows<__nv_bfloat16, KIND, GRAD>(a, (cudaStream_t)stream)
                                     : choose_rows<float, KIND, GRAD>(a, (cudaStream_t)stream);
}

int logp_forward(const bf16opt_tokens_t *d, float *logp, float *saved, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check_tokens(d);
    if (rc != BF16OPT_OK) return rc;
    rc = check(d, {}, {{logp, d->rows * 4}, {saved, d->rows * 16}}, nullptr, 0, false);
    if (rc != BF16OPT_OK || d->rows == 0) return rc;
    if (!logp) return bad("an output pointer is NULL");
    if (misaligned(saved, 16)) return fail(BF16OPT_ERR_ALIGNMENT, "logp: saved must be 16-byte aligned");
    Args a = args_of(d);
    a.logp = logp, a.saved = reinterpret_cast<float4 *>(saved);
    return rows_kernel<LOGP, false>(a, d->logits_type, stream);
}

int logp_backward(const bf16opt_tokens_t *d, const float *saved, const float *dloss, uint64_t losses, void *dlogits, uint64_t dlogits_stride, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check_tokens(d);
    if (rc != BF16OPT_OK) return rc;
    if (losses > BF16OPT_TOKENS_MAX_ROWS) return bad("losses exceeds BF16OPT_TOKENS_MAX_ROWS");
    rc = check(d, {{saved, d->rows * 16}, {dloss, losses * 4}}, {}, dlogits, dlogits_stride, true);
    if (rc != BF16OPT_OK || d->rows == 0) return rc;
    if (!saved) return bad("saved is NULL");
    if (misaligned(saved, 16)) return fail(BF16OPT_ERR_ALIGNMENT, "logp: saved must be 16-byte aligned");
    if (sm_count() < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "logp: no CUDA device");
    Args a = args_of(d);
    a.saved_in = reinterpret_cast<const float4 *>(saved);
    a.dloss = dloss, a.losses = losses, a.dlogits = dlogits, a.dlogits_stride = dlogits_stride;
    const uint64_t vecs = d->vocab / (16 / type_bytes(d->logits_type));
    a.slices = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(1, vecs / kSliceVectors), 0x7fffffffu / d->rows);
    const Launch l{(unsigned)(a.rows * a.slices), kThreads, 0, (cudaStream_t)stream, 0, true};
    const cudaError_t e = d->logits_type == BF16OPT_TYPE_BF16 ? launch(l, k_backward<__nv_bfloat16>, a) : launch(l, k_backward<float>, a);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "logp kernel launch");
}

int check_policy(const bf16opt_tokens_t *d, const bf16opt_policy_t *p) {
    const int rc = check_tokens(d);
    if (rc != BF16OPT_OK) return rc;
    if (!p) return bad("the policy's descriptor is NULL");
    if (!(p->clip_low >= 0.f && p->clip_low <= 1.f) || !(p->clip_high >= 0.f)) return bad("clip_low must lie in [0, 1], clip_high be >= 0");
    if (!(std::isfinite(p->kl_weight) && p->kl_weight >= 0.f)) return bad("kl_weight must be finite and >= 0");
    if (p->reserved) return bad("reserved must be 0");
    return BF16OPT_OK;
}

template <bool GRAD>
int policy(const bf16opt_tokens_t *d, const bf16opt_policy_t *p, const float *dloss, float *loss, float *logp, float *saved, void *dlogits,
           uint64_t dlogits_stride, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check_policy(d, p);
    if (rc != BF16OPT_OK) return rc;
    const uint64_t r4 = d->rows * 4;
    rc = check(d, {{p->advantage, r4}, {p->old_logp, r4}, {p->ref_logp, r4}, {dloss, r4}}, {{loss, r4}, {logp, r4}, {saved, 4 * r4}}, dlogits,
               dlogits_stride, GRAD);
    if (rc != BF16OPT_OK || d->rows == 0) return rc;
    if (!loss || !p->advantage || (!GRAD && !logp)) return bad("a pointer is NULL");
    if (misaligned(saved, 16)) return fail(BF16OPT_ERR_ALIGNMENT, "logp: saved must be 16-byte aligned");
    Args a = args_of(d);
    a.advantage = p->advantage, a.old_logp = p->old_logp, a.ref_logp = p->kl_weight != 0.f ? p->ref_logp : nullptr;
    a.lowest = 1.f - p->clip_low, a.highest = 1.f + p->clip_high, a.kl_weight = p->kl_weight;
    a.dloss = dloss, a.loss = loss, a.logp = logp, a.saved = reinterpret_cast<float4 *>(saved);
    a.dlogits = dlogits, a.dlogits_stride = dlogits_stride;
    return rows_kernel<POLICY, GRAD>(a, d->logits_type, stream);
}

int preference(const bf16opt_tokens_t *d, const bf16opt_preference_t *p, float *loss, float *logp, float *saved, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    int rc = check_tokens(d);
    if (rc != BF16OPT_OK) return rc;
    if (!p) return bad("the preference's descriptor is NULL");
    if (!index_ok(p->offsets_type)) return bad("unknown index type");
    if (p->kind != BF16OPT_PREFER_SIGMOID && p->kind != BF16OPT_PREFER_HINGE && p->kind != BF16OPT_PREFER_IPO) return bad("unknown kind of loss");
    if (p->pairs > BF16OPT_PREFER_MAX_PAIRS) return bad("pairs exceeds BF16OPT_PREFER_MAX_PAIRS");
    if (!(std::isfinite(p->beta) && p->beta > 0.f) || !std::isfinite(0.5f / p->beta)) return bad("beta must be finite and > 0");
    if (!(p->label_smoothing >= 0.f && p->label_smoothing <= 0.5f)) return bad("label_smoothing must lie in [0, 0.5]");
    if (!std::isfinite(p->margin)) return bad("margin must be finite");
    if (p->length_normalise != 0 && p->length_normalise != 1) return bad("length_normalise must be 0 or 1");
    if (d->row_weight) return bad("row_weight must be NULL: labels say which rows count");
    const uint64_t pairs = p->pairs, ib = index_bytes(p->offsets_type);
    if (pairs && (!p->offsets || !loss || !logp)) return bad("a pointer is NULL");
    if (pairs && misaligned(p->offsets, ib)) return fail(BF16OPT_ERR_ALIGNMENT, "logp: a pointer is not aligned to its element");
    rc = check(d, {{p->offsets, (2 * pairs + 1) * ib}, {p->ref_logp, pairs * 8}}, {{loss, pairs * 4}, {logp, pairs * 8}, {saved, d->rows * 16}}, nullptr, 0, false);
    if (rc != BF16OPT_OK) return rc;
    if (d->rows && !saved) return bad("saved is NULL");
    if (misaligned(saved, 16) || misaligned(loss, 4) || misaligned(logp, 4) || misaligned(p->ref_logp, 4))
        return fail(BF16OPT_ERR_ALIGNMENT, "logp: saved must be 16-byte aligned, FP32 arrays to their element");
    Args a = args_of(d);
    a.offsets = p->offsets, a.offsets_type = p->offsets_type, a.pairs = pairs;
    a.loss = loss, a.logp = logp, a.saved = reinterpret_cast<float4 *>(saved);
    if (d->rows) {
        rc = rows_kernel<PREFER, false>(a, d->logits_type, stream);
        if (rc != BF16OPT_OK) return rc;
    }
    if (!pairs) return BF16OPT_OK;
    if (sm_count() < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "logp: no CUDA device");
    PairArgs q = {a, p->kind, p->length_normalise, p->beta, p->label_smoothing, p->margin, 0.5 / (double)p->beta, p->ref_logp};
    const Launch l{(unsigned)pairs, kPairThreads, 0, (cudaStream_t)stream, 0, true};
    const cudaError_t e = d->logits_type == BF16OPT_TYPE_BF16 ? launch(l, k_pairs<__nv_bfloat16>, q) : launch(l, k_pairs<float>, q);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "logp kernel launch");
}

}  // namespace
}  // namespace bf16ops

extern "C" int bf16opt_token_logp_forward(const bf16opt_tokens_t *d, float *logp, float *saved, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::logp_forward(d, logp, saved, stream); });
}

extern "C" int bf16opt_token_logp_backward(const bf16opt_tokens_t *d, const float *saved, const float *dloss, uint64_t losses,
                                           void *dlogits, uint64_t dlogits_stride, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::logp_backward(d, saved, dloss, losses, dlogits, dlogits_stride, stream); });
}

extern "C" int bf16opt_policy_forward(const bf16opt_tokens_t *d, const bf16opt_policy_t *p, float *loss, float *logp, float *saved, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::policy<false>(d, p, nullptr, loss, logp, saved, nullptr, 0, stream); });
}

extern "C" int bf16opt_policy_loss_grad(const bf16opt_tokens_t *d, const bf16opt_policy_t *p, const float *dloss, float *loss, float *logp,
                                        void *dlogits, uint64_t dlogits_stride, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::policy<true>(d, p, dloss, loss, logp, nullptr, dlogits, dlogits_stride, stream); });
}

extern "C" int bf16opt_preference_forward(const bf16opt_tokens_t *d, const bf16opt_preference_t *p, float *loss, float *logp, float *saved, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::preference(d, p, loss, logp, saved, stream); });
}
