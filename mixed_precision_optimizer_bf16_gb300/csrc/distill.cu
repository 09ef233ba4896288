// distill.cu -- distillation from a teacher's top logits, forward and backward
// (bf16opt_distill_* of include/bf16opt.h).
//
// A row's loss needs the log-sum-exp of its logits and its gradient needs the
// logits again.  A cluster of CTAs (often of one) takes a row: each CTA streams its
// slice of the row once, keeping a running maximum and sums per thread; the CTAs' sums meet
// through distributed shared memory; then each CTA writes its slice's gradient,
// from what it kept of the slice in shared memory and, for the rest, from L2.  Every logit is
// so read from HBM about once and every gradient written once: 4 bytes per bf16
// logit, which is what bounds the operator (with two temperatures, the
// special-function unit comes next).
//
// The teacher's k entries of a row (and the label, as one more entry) are held
// in shared memory by every CTA of the cluster.  Their softmax is computed by
// each CTA by itself, and their part of the gradient is put on top of the
// slice's: an entry's element is recomputed and stored again with everything
// that its id collects, rounded once.
//
// Measured on one GB300 (algorithmic bytes over the time; a copy of the same
// buffers runs at 6.75 TB/s), bf16 logits with 64 entries: 2048 rows of 250880 with
// labels, T = 2, loss and gradient 422 us, 4.9 TB/s; at T = 1 without labels 1024 rows of 250880
// forward 90 us, 5.7 TB/s, backward 175 us, 5.9 TB/s; 8192 rows of 32000 forward 108 us, 4.8 TB/s,
// backward 177 us, 5.9 TB/s, loss and gradient 209 us, 5.0 TB/s (241 us with labels at T = 2).
// At 250880 the two-pass kernel reads 51 % more from DRAM than the operator needs, what did not stay
// in its ring and misses L2 (22 % more bytes in all), which is most of its time; it issues in
// 59 % of the slots.  Small rows are bound by the latency of a row's reductions.
#include <cooperative_groups.h>

#include <algorithm>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace bf16ops {
namespace {

// Vectors of a thread in a group of the ring.  8 gave 220 against 231 us at T = 1.5 on 1024 x
// 250880, but 317 against 226 us on 8192 x 32000 (a row is then less than two groups).
constexpr int kU = 4;
constexpr int kMaxCluster = 8;
// Threads of a CTA: of the kernels with one pass, and with both where rows are short (up to
// kShortRow vectors); and with both where they are long, which wants more than 80 registers:
// 1024 x 250880 took 256 us with 384 threads at 80 registers, 214 us so.
constexpr int kSmall = 192, kLarge = 256;
constexpr uint64_t kShortRow = 5000;
// CTAs of an SM, and groups in the ring of each, by their threads: 200 KB of an SM are rings.
__host__ __device__ constexpr int resident(int threads) { return threads == kLarge ? 2 : 4; }
__host__ __device__ constexpr int ring_depth(int threads) { return 200 * 1024 / resident(threads) / (threads * kU * 16); }
// Saved log-sum-exps below this are taken as they are: their rounding is at most 2^-18, which is how far it
// moves a softmax, as much as the exponents' own.
constexpr float kFar = 128.f;
// Entries of one thread, the label's included.
__host__ __device__ constexpr int entries(int threads) { return (BF16OPT_DISTILL_MAX_K + threads) / threads; }

struct Args {
    uint64_t rows;
    uint32_t vocab, k;
    int teacher_type, ids_type, labels_type;
    const void *logits;
    uint64_t logits_stride;
    const void *ids;
    uint64_t ids_stride;
    const void *teacher;
    uint64_t teacher_stride;
    const float *teacher_lse;
    const void *labels;
    const float *row_weight;
    float inv_t;                      // 1 / temperature
    float temperature;
    float kl_weight, ce_weight;       // ce_weight 0 without labels
    const float *dloss;
    const float *lse_in;
    float *loss, *lse_out;
    void *dlogits;
    uint64_t dlogits_stride;
};

// Running softmax of a stream of numbers: their maximum, and the sums of
// exp((z - max) / T) and of exp(z - max).
struct Stat {
    float m, st, s1;
};
// The teacher's: maximum m of t, sum s of e = exp((t - m) / T), sum d of e ((t - m) / T - (z - b) / T),
// b the largest finite z: both taken from their largest before anything is rounded, so that logits far
// from 0 cost no digits.
struct Teach {
    float m, b, s, d;
};

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.f : m; }

// y - m / T, where both are large and near one another: with the quotient's rounding error.
__device__ __forceinline__ float less_quotient(float y, float m, float inv_t, float t) {
    const float q = m * inv_t;
    return fabsf(q) < INFINITY ? (y - q) - fmaf(-q, t, m) * inv_t : y - q;
}

// Each product and sum rounded by itself, so that join(a, b) and join(b, a) are the same bits.
__device__ __forceinline__ float weighted(float a, float ea, float b, float eb) {
    return __fadd_rn(__fmul_rn(a, ea), __fmul_rn(b, eb));
}
template <int POWER>
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b, float c_t) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    const float m = safe_max(r.m);
    r.st = weighted(a.st, ex2((a.m - m) * c_t), b.st, ex2((b.m - m) * c_t));
    r.s1 = POWER ? weighted(a.s1, ex2((a.m - m) * kLog2e), b.s1, ex2((b.m - m) * kLog2e)) : 0.f;
    return r;
}
// Joined over the warp: first the maximum, then the sums scaled to it, so that
// a step is a shuffle and one operation; every lane gets the same bits.
template <int POWER>
__device__ __forceinline__ Stat warp_join(const Stat &a, float c_t) {
    Stat r;
    r.m = warp_max(a.m);
    const float d = a.m - safe_max(r.m);
    r.st = warp_sum(a.st * ex2(d * c_t));
    r.s1 = POWER ? warp_sum(a.s1 * ex2(d * kLog2e)) : 0.f;
    return r;
}
__device__ __forceinline__ Teach warp_join(const Teach &a, float inv_t) {
    Teach r;
    r.m = warp_max(a.m);
    r.b = warp_max(a.b);
    const float x = (a.m - safe_max(r.m)) * inv_t, e = ex2(x * kLog2e);
    r.s = warp_sum(a.s * e);
    // a d of +inf (masked z) may meet a weight of 0
    r.d = warp_sum(e > 0.f ? e * (a.d + a.s * (x - (safe_max(a.b) - safe_max(r.b)) * inv_t)) : 0.f);
    return r;
}

// exp(d) from e = exp(d / T): T = POWER (2 or 4) by squaring.
template <int POWER>
__device__ __forceinline__ float2 powered(float2 e) {
    const float2 q = mul2(e, e);
    return POWER == 4 ? mul2(q, q) : q;
}

// The exponents (z - m) c of a softmax in base 2.  The difference is formed first: exact near the top,
// wherever the row lies.  (As z c - m c in one instruction the rounded product is off in every term,
// 2e-6 of a loss at m = 20, overflows where the logits are the type's lowest, and no call was faster.)
__device__ __forceinline__ float2 exponent(float2 z, float m, float c) { return mul2(add2(z, both(-m)), both(c)); }

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

// Slots of the table of ids: a power of two, at least twice the entries.
__host__ __device__ constexpr uint32_t table_size(uint32_t k) {
    uint32_t n = 4;
    while (n < 2 * (k + 1)) n *= 2;
    return n;
}

// A row whose saved log-sum-exps do not say enough for its gradient: one FP32 number has no room for the sum's
// logarithm beside a far maximum, or is infinite (where every logit is masked, too).
__device__ __forceinline__ bool is_far(const Args &a, float lse_t, float lse_1) {
    return !(fabsf(lse_t) < kFar && fabsf(lse_1) < kFar && fabsf(lse_t * a.temperature) < INFINITY);
}

// FORWARD: the row's sums are computed here (else read from lse_in).  GRAD: the
// gradient is written.  POWER: 0, only the softmax at T is needed; 1, the one at
// temperature 1 too; 2 or 4, the same with T = POWER, where exp(d) is a power
// of exp(d / T) -- the special-function unit is what such a row is short of.
//
// A slice passes through a ring of shared memory, `depth` groups of kU vectors
// of every thread.  A slot is touched by one thread alone, so no barrier guards
// it: the thread copies its vectors in asynchronously, waits for its own copies
// and, after the last use, copies in what comes `depth` groups later -- of this row
// or of the cluster's next ones.  With both passes (FORWARD and GRAD) the slice's last
// `depth` groups stay in the ring for the gradient, which starts with them; the ones
// before are read a second time, from L2, where the row still is.
//
// Without FORWARD far rows are passed over. FAR: those rows alone, their sums computed once more, and no loss
// written: the second launch of the backward call, over at once where there are none.  (With the sums of far rows
// in one kernel, in any place of it, registers spilled: 1024 x 250880 bf16 241 to 249 us, 1021 x 32003 FP32 62 to
// 69 us, so 181 and 58 us, 178 and 55 us without the second launch.)
template <int kThreads, class T, bool FORWARD, bool GRAD, int POWER, bool FAR = false>
__global__ void __launch_bounds__(kThreads, resident(kThreads)) k_distill(const Args a) {
    constexpr int N = Vec<T>::N, P = N / 2;
    constexpr uint32_t kGroup = kThreads * kU, depth = ring_depth(kThreads);
    constexpr int kWarps = kThreads / 32, kEntries = entries(kThreads);
    // 128 bytes: a ring that begins elsewhere splits every wavefront (1024 x 250880 forward, 80 bytes
    // off: 108 against 88 us)
    extern __shared__ __align__(128) unsigned char smem_raw[];
    // ring | ids, t (then what the entry takes off the gradient), z of the entries
    uint4 *ring = reinterpret_cast<uint4 *>(smem_raw);
    int32_t *sm_id = reinterpret_cast<int32_t *>(smem_raw + (size_t)depth * kGroup * 16);
    float *sm_x = reinterpret_cast<float *>(sm_id + (a.k + 1));
    float *sm_z = sm_x + (a.k + 1);
    int32_t *sm_table = reinterpret_cast<int32_t *>(sm_z + (a.k + 1));   // GRAD: [table_size(k)], ids of the slice's entries
    __shared__ Stat sm_stat[2][kMaxCluster * kWarps];   // [turn][rank][warp]
    __shared__ Teach sm_teach[2][kWarps];
    __shared__ uint32_t sm_twice[2];      // the last turn of that parity in which an id came twice
    __shared__ int32_t sm_label[2];
    __shared__ float sm_label_z[2];

    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t log2_ranks = 31 - __clz(ranks);   // a power of two
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t n_entries = a.k + 1;   // the label is the last one, thread kThreads - 1's
    const float c_t = a.inv_t * kLog2e;
    const uint64_t step = gridDim.x / ranks;
    const uint32_t table = table_size(a.k);
    if (GRAD) {
        for (uint32_t i = tid; i < table; i += kThreads) sm_table[i] = -1;
        if (tid < 2) sm_twice[tid] = 0;
        __syncthreads();
    }
    pdl_enter();
    if constexpr (FAR) {
        bool any = false;
        for (uint64_t r = blockIdx.x / ranks + tid * step; r < a.rows; r += kThreads * step) any |= is_far(a, a.lse_in[2 * r], a.lse_in[2 * r + 1]);
        if (!__syncthreads_or(any)) return;   // the same in every CTA of the cluster
    }
    if (FORWARD && ranks > 1) cluster.sync();   // every CTA's shared memory exists

    auto row_of = [&](uint64_t row) { return reinterpret_cast<const T *>(a.logits) + row * a.logits_stride; };
    auto weight_of = [&](uint64_t row) {
        if (row >= a.rows || (FAR && !is_far(a, a.lse_in[2 * row], a.lse_in[2 * row + 1]))) return 0.f;
        return a.row_weight ? a.row_weight[row] : 1.f;
    };
    // Entry `tid` of a row (of thread kThreads - 1 the label, where it has no entry; further
    // entries when they are needed): its id and logit are asked for two rows ahead, the student's
    // logit at the id one row ahead.
    struct Entry {
        int64_t id;
        float t;
    };
    auto fetch_entry = [&](uint64_t row, float w) {
        Entry e = {-1, 0.f};
        if (w != 0.f && tid < a.k) {
            e.id = load_index(a.ids, a.ids_type, row * a.ids_stride + tid);
            e.t = load_typed(a.teacher, a.teacher_type, row * a.teacher_stride + tid);
        } else if (w != 0.f && tid == kThreads - 1 && a.ce_weight != 0.f && a.k < kThreads) {
            e.id = load_index(a.labels, a.labels_type, row);
        }
        return e;
    };
    auto fetch_z = [&](uint64_t row, const Entry &e) { return e.id >= 0 && e.id < (int64_t)a.vocab ? to_f32(row_of(row)[e.id]) : 0.f; };
    // a row's numbers, asked for one row ahead
    struct Scalars {
        float up, teacher_lse, lse_t, lse_1;
    };
    auto scalars_of = [&](uint64_t row) {
        Scalars v = {1.f, 0.f, 0.f, 0.f};
        if (row < a.rows) {
            if (GRAD && a.dloss) v.up = a.dloss[row];
            if (a.teacher_lse) v.teacher_lse = a.teacher_lse[row];
            if (!FORWARD) v.lse_t = a.lse_in[2 * row], v.lse_1 = a.lse_in[2 * row + 1];
        }
        return v;
    };

    uint64_t row = blockIdx.x / ranks;
    float w = weight_of(row), w_next = weight_of(row + step);
    Scalars now = scalars_of(row);
    Entry entry = fetch_entry(row, w), entry_next = fetch_entry(row + step, w_next);
    float entry_z = fetch_z(row, entry);
    // What is copied into the ring next: group `i` of `n` of a row's slice.
    struct Cursor {
        uint64_t row;
        const uint4 *zv;
        uint32_t nv, n, i;
        bool again;        // the groups that did not stay, for the gradient
        float w, w_next;
    } cur = {};
    auto open_row = [&]() {   // the first row from cur.row on that is read at all
        while (cur.row < a.rows && cur.w == 0.f) cur.row += step, cur.w = cur.w_next, cur.w_next = weight_of(cur.row + step);
        if (cur.row < a.rows) {
            const Slice s = slice_of(row_of(cur.row), a.vocab, rank, ranks, log2_ranks);
            cur.zv = reinterpret_cast<const uint4 *>(row_of(cur.row) + s.head) + s.v0 + tid;
            cur.nv = s.v1 - s.v0;
            cur.n = max(1u, (cur.nv + kGroup - 1) / kGroup);
            cur.i = 0;
            cur.again = false;
        }
    };
    uint32_t issued = 0, issued_slot = 0;
    auto issue = [&]() {
        if (cur.row < a.rows) {
            uint4 *to = ring + issued_slot * kGroup + tid;
            const uint4 *from = cur.zv + cur.i * kGroup;
            if ((cur.i + 1) * kGroup <= cur.nv) {
#pragma unroll
                for (int u = 0; u < kU; ++u) copy_async16(to + u * kThreads, from + u * kThreads);
            } else {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (cur.i * kGroup + u * kThreads + tid < cur.nv) copy_async16(to + u * kThreads, from + u * kThreads);
            }
            ++cur.i;
            const bool over = cur.i == (cur.again ? cur.n - depth : cur.n);
            if (over && FORWARD && GRAD && !cur.again && cur.n > depth) {
                cur.again = true;
                cur.i = 0;
            } else if (over) {
                cur.row += step, cur.w = cur.w_next, cur.w_next = weight_of(cur.row + step);
                open_row();
            }
        }
        copy_commit();
        ++issued;
        issued_slot = issued_slot + 1 == depth ? 0 : issued_slot + 1;
    };
    cur.row = row, cur.w = w, cur.w_next = w_next;
    open_row();
    for (uint32_t i = 0; i < depth; ++i) issue();
    uint32_t seen = 0, slot = 0;   // groups of the ring that have been waited for, and the slot of the next
    // the next group of the ring, once it is there: `full` without looking at the slice's end
    auto take = [&](uint4 (&q)[kU], uint32_t i, uint32_t nv) {
        copy_wait_for(issued - 1 - seen);
        const uint4 *from = ring + slot * kGroup + tid;
        const bool full = (i + 1) * kGroup <= nv;
        if (full) {
#pragma unroll
            for (int u = 0; u < kU; ++u) q[u] = from[u * kThreads];
        } else {
#pragma unroll
            for (int u = 0; u < kU; ++u) q[u] = i * kGroup + u * kThreads + tid < nv ? from[u * kThreads] : nothing<T>();
        }
        ++seen;
        slot = slot + 1 == depth ? 0 : slot + 1;
    };

    uint32_t turn = 1;
    for (; row < a.rows; row += step) {
        const T *z = row_of(row);
        T *out = GRAD ? reinterpret_cast<T *>(a.dlogits) + row * a.dlogits_stride : nullptr;
        const Slice s = slice_of(z, a.vocab, rank, ranks, log2_ranks);
        const bool whole = GRAD && (((uintptr_t)out ^ (uintptr_t)z) & 15u) == 0;
        const uint4 *zv = reinterpret_cast<const uint4 *>(z + s.head) + s.v0;
        T *ov = GRAD ? out + s.head + (size_t)s.v0 * N : nullptr;
        const uint32_t nv = s.v1 - s.v0;
        const uint32_t n = max(1u, (nv + kGroup - 1) / kGroup), stay = n > depth ? n - depth : 0u;   // groups from `stay` on stay
        const uint64_t next = row + step;
        const float w_after = weight_of(next + step);
        const Scalars then = scalars_of(next);

        if (w == 0.f) {   // not read: zeros (which the first launch has written where FAR)
            if (GRAD && !FAR) {
                float zero[N] = {};
                for (uint32_t j = tid; j < nv; j += kThreads) store_vec<T>(ov + (size_t)j * N, zero, whole);
                if (rank == 0 && tid < s.head) from_f32(out[tid], 0.f);
                if (rank + 1 == ranks && tid < a.vocab - s.tail0) from_f32(out[s.tail0 + tid], 0.f);
            }
            if (FORWARD && !FAR && rank == 0 && tid == 0) {
                a.loss[row] = 0.f;
                if (a.lse_out) a.lse_out[2 * row] = a.lse_out[2 * row + 1] = 0.f;
            }
            w = w_next, w_next = w_after, now = then;
            entry = entry_next, entry_next = fetch_entry(next + step, w_next);
            entry_z = fetch_z(next, entry);
            continue;
        }

        const Entry entry_after = fetch_entry(next + step, w_after);
        const float z_next = fetch_z(next, entry_next);
        const float up = w * now.up, wr = w;

        // ---- the slice's running maximum and sums
        Stat st = {-INFINITY, 0.f, 0.f};
        if (FORWARD) {
            float2 sum_t = both(0.f), sum_1 = both(0.f);
            for (uint32_t i = 0; i < n; ++i) {
                uint4 q[kU];
                take(q, i, nv);
                const float mx = largest<T, kU>(q);
                if (mx > st.m) {   // the sums move to the new maximum (the first time from -inf: by 0)
                    sum_t = mul2(sum_t, both(ex2((st.m - mx) * c_t)));
                    if (POWER) sum_1 = mul2(sum_1, both(ex2((st.m - mx) * kLog2e)));
                    st.m = mx;
                }
                const float m = safe_max(st.m);
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    float2 f[P];
                    pairs<T>(q[u], f);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const float2 d = exponent(f[i], m, c_t);
                        const float2 e = make_float2(ex2(d.x), ex2(d.y));
                        sum_t = add2(sum_t, e);
                        if (POWER == 1) {
                            const float2 d1 = exponent(f[i], m, kLog2e);
                            sum_1 = add2(sum_1, make_float2(ex2(d1.x), ex2(d1.y)));
                        } else if (POWER > 1) {
                            sum_1 = add2(sum_1, powered<POWER>(e));
                        }
                    }
                }
                if (!GRAD || i < stay) issue();
            }
            st.st = sum_t.x + sum_t.y;
            st.s1 = sum_1.x + sum_1.y;
            uint32_t at = 0xffffffffu;
            if (rank == 0 && tid < s.head) at = tid;
            else if (rank + 1 == ranks && tid >= 32 && tid - 32 < a.vocab - s.tail0) at = s.tail0 + tid - 32;
            if (at != 0xffffffffu) {
                const float f = to_f32(z[at]);
                const float one = f == -INFINITY ? 0.f : f == f ? 1.f : f;   // a NaN stays one
                st = join<POWER>(st, Stat{f == f ? f : -INFINITY, one, one}, c_t);
            }
        }

        // ---- the entries' softmax
        Teach te = {-INFINITY, -INFINITY, 0.f, 0.f};
        uint32_t slots[kEntries];   // where this thread's entries stand in the table
#pragma unroll
        for (int i = 0; i < kEntries; ++i) slots[i] = 0xffffffffu;
        // An id of the slice goes into an open table; one that is there already has come twice.
        auto enter = [&](int32_t id) -> uint32_t {
            if (!GRAD || id < (int32_t)s.lo || id >= (int32_t)s.hi) return 0xffffffffu;
            uint32_t at = (uint32_t)id * 2654435761u & (table - 1);
            for (uint32_t n = 0; n < table; ++n) {
                const int32_t was = atomicCAS(&sm_table[at], -1, id);
                if (was == -1) return at;
                if (was == id) break;
                at = (at + 1) & (table - 1);
            }
            sm_twice[turn & 1] = turn;
            return 0xffffffffu;
        };
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
            const uint32_t e = tid + i * kThreads;
            if (e >= a.k) break;
            const int64_t id64 = i == 0 ? entry.id : load_index(a.ids, a.ids_type, row * a.ids_stride + e);
            const float t = i == 0 ? entry.t : load_typed(a.teacher, a.teacher_type, row * a.teacher_stride + e);
            const bool there = id64 >= 0 && id64 < (int64_t)a.vocab && t != -INFINITY;
            const int32_t id = there ? (int32_t)id64 : -1;
            const float zi = i == 0 ? entry_z : there ? to_f32(z[id]) : 0.f;
            sm_id[e] = id, sm_x[e] = t, sm_z[e] = zi;
            if (there) {
                te.m = fmaxf(te.m, t);
                if (fabsf(zi) < INFINITY) te.b = fmaxf(te.b, zi);
            }
            slots[i] = enter(id);
        }
        if (tid == kThreads - 1) {   // the label, entry a.k
            int64_t id64 = -1;
            float zi = entry_z;
            if (a.ce_weight != 0.f) {
                id64 = entry.id;
                if (a.k >= kThreads) {   // this thread had an entry to fetch
                    id64 = load_index(a.labels, a.labels_type, row);
                    zi = id64 >= 0 && id64 < (int64_t)a.vocab ? to_f32(z[id64]) : 0.f;
                }
            }
            const int32_t id = id64 >= 0 && id64 < (int64_t)a.vocab ? (int32_t)id64 : -1;
            sm_id[a.k] = sm_label[turn & 1] = id;
            sm_z[a.k] = sm_label_z[turn & 1] = zi;
            slots[kEntries - 1] = enter(id);
        }
        entry = entry_next, entry_next = entry_after, entry_z = z_next;
        w = w_next, w_next = w_after;

        // ---- joined over the warp, and the warps of the cluster (CTA) in one step
        const uint32_t teach_warps = min((uint32_t)kWarps, (a.k + 31) / 32);
        if (warp < teach_warps) {   // (both, so that their shuffles run side by side)
            te.m = warp_max(te.m), te.b = warp_max(te.b);
            for (uint32_t i = tid; i < a.k; i += kThreads) {   // its own entries
                const float x = (sm_x[i] - safe_max(te.m)) * a.inv_t, e = sm_id[i] < 0 ? 0.f : ex2(x * kLog2e);
                te.s += e;
                if (!(e <= 0.f)) te.d += e * (x - (sm_z[i] - safe_max(te.b)) * a.inv_t);
            }
            te.s = warp_sum(te.s), te.d = warp_sum(te.d);
            if (FORWARD) st = warp_join<POWER>(st, c_t);
            if (lane == 0) sm_teach[turn & 1][warp] = te;
        } else if (FORWARD) {
            st = warp_join<POWER>(st, c_t);
        }
        if (FORWARD) {
            if (lane < ranks) {
                Stat *to = &sm_stat[turn & 1][rank * kWarps + warp];
                *(ranks > 1 ? cluster.map_shared_rank(to, lane) : to) = st;
            }
        }
        if (FORWARD && ranks > 1) cluster.sync();
        else __syncthreads();
        if (!GRAD && (rank != 0 || warp != 0)) {   // the loss is one warp's
            now = then;
            ++turn;
            continue;
        }
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (slots[i] != 0xffffffffu) sm_table[slots[i]] = -1;   // everybody's are in: for the next row
        te = lane < teach_warps ? sm_teach[turn & 1][lane] : Teach{-INFINITY, -INFINITY, 0.f, 0.f};
        te = warp_join(te, a.inv_t);
        float lse_t, lse_1, log_t, log_1;   // lse_t = m / T + log_t, lse_1 = m + log_1
        bool empty;   // no logit but -inf in the row
        // q = exp2((z - base_t) c_t) exp2(rest_t): the base near the row's top, so that z - base is exact there
        float base_t, rest_t, base_1, rest_1;
        if (FORWARD) {
            st = lane < ranks * kWarps ? sm_stat[turn & 1][lane] : Stat{-INFINITY, 0.f, 0.f};
            for (uint32_t i = lane + 32; i < ranks * kWarps; i += 32) st = join<POWER>(st, sm_stat[turn & 1][i], c_t);
            st = warp_join<POWER>(st, c_t);
            const float m = safe_max(st.m);
            empty = st.m == -INFINITY && st.st == 0.f;
            log_t = logf(st.st);
            log_1 = POWER ? logf(st.s1) : log_t;
            lse_t = empty ? -INFINITY : m * a.inv_t + log_t;
            lse_1 = empty ? -INFINITY : (POWER ? m + log_1 : lse_t);
            base_t = base_1 = m;
            rest_t = empty ? 0.f : -log2f(st.st);
            rest_1 = POWER && !empty ? -log2f(st.s1) : 0.f;
        } else {
            lse_t = now.lse_t;
            lse_1 = now.lse_1;
            empty = false;
            base_t = lse_t * a.temperature;
            rest_t = fmaf(lse_t, a.temperature, -base_t) * -c_t;
            base_1 = lse_1;
            rest_1 = 0.f;
        }

        // ---- the row's loss
        const bool some = te.s != 0.f;   // the teacher has entries here (NaN counts)
        const float log_teacher = a.teacher_lse ? less_quotient(now.teacher_lse, te.m, a.inv_t, a.temperature) : logf(te.s);   // the lse less te.m / T
        const float mass = !some ? 0.f : a.teacher_lse ? te.s * ex2(-log_teacher * kLog2e) : te.s == te.s ? 1.f : te.s;
        const bool has_label = sm_label[turn & 1] >= 0;
        const bool skip = !FORWARD && is_far(a, now.lse_t, now.lse_1);   // its gradient is the second launch's
        now = then;
        if (FORWARD && !FAR && rank == 0 && tid == 0) {
            float kl = 0.f, ce = 0.f;
            if (some && a.kl_weight != 0.f && mass != 0.f)
                kl = empty ? INFINITY
                           : a.kl_weight * a.temperature * a.temperature * mass *
                                 (te.d / te.s + ((base_t - safe_max(te.b)) * a.inv_t + log_t) - log_teacher);
            if (has_label) ce = empty ? INFINITY : a.ce_weight * ((base_t - sm_label_z[turn & 1]) + log_1);
            a.loss[row] = wr * (kl + ce);
            if (a.lse_out) a.lse_out[2 * row] = lse_t, a.lse_out[2 * row + 1] = lse_1;
        }
        if (!GRAD) {
            ++turn;
            continue;
        }

        // ---- the gradient of the slice
        const float hard = has_label ? up * a.ce_weight : 0.f;
        const float soft = up * a.kl_weight * a.temperature;
        // T = POWER: exp2((z - base_1) log2e + rest_1) = e^POWER exp2(shift), e the value at T; e <= 1 and the
        // factor stays with it (where a factor overflows, the top's own e is as small as the factor is large)
        const float shift = POWER > 1 ? (base_t - base_1) * kLog2e + rest_1 : rest_1;
        // both terms have the same softmax where POWER is 0
        const float a_t = (soft * mass + (POWER ? 0.f : hard)) * ex2(rest_t), a_1 = POWER ? hard * ex2(shift) : 0.f;
        auto grad2 = [&](float2 f) {
            const float2 d = exponent(f, base_t, c_t);
            const float2 e = make_float2(ex2(d.x), ex2(d.y));
            float2 g = mul2(both(a_t), e);
            if (POWER == 1) {
                const float2 d1 = exponent(f, base_1, kLog2e);
                g = fma2(both(a_1), make_float2(ex2(d1.x), ex2(d1.y)), g);
            } else if (POWER > 1) {
                g = fma2(both(a_1), powered<POWER>(e), g);
            }
            return g;
        };
        auto grad = [&](float f) { return grad2(make_float2(f, f)).x; };
        auto grad_group = [&](const uint4 (&q)[kU], uint32_t i) {
            const bool full = (i + 1) * kGroup <= nv;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const uint32_t j = i * kGroup + u * kThreads + tid;
                if (!full && j >= nv) break;
                float2 f[P];
                pairs<T>(q[u], f);
                float g[N];
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const float2 r = grad2(f[k]);
                    g[2 * k] = r.x, g[2 * k + 1] = r.y;
                }
                store_vec<T>(ov + (size_t)j * N, g, whole);
            }
        };
        if (FORWARD) {   // the groups that stayed: the last ones seen
            uint32_t at = n - stay > slot ? slot + depth - (n - stay) : slot - (n - stay);
            for (uint32_t i = stay; i < n; ++i) {
                const uint4 *from = ring + at * kGroup + tid;
                uint4 q[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) q[u] = from[u * kThreads];
                at = at + 1 == depth ? 0 : at + 1;
                grad_group(q, i);
                issue();
            }
        }
        for (uint32_t i = 0; i < (FORWARD ? stay : n); ++i) {
            uint4 q[kU];
            take(q, i, nv);
            if (!skip) grad_group(q, i);
            issue();
        }
        if (rank == 0 && tid < s.head && !skip) from_f32(out[tid], grad(to_f32(z[tid])));
        if (rank + 1 == ranks && tid < a.vocab - s.tail0 && !skip)
            from_f32(out[s.tail0 + tid], grad(to_f32(z[s.tail0 + tid])));

        // ---- the entries of the slice
        const bool twice = sm_twice[turn & 1] == turn;
        ++turn;
        for (uint32_t e = tid; e < a.k; e += kThreads) sm_x[e] = soft * ex2(((sm_x[e] - te.m) * a.inv_t - log_teacher) * kLog2e);
        if (tid == kThreads - 1) sm_x[a.k] = hard;
        __syncthreads();   // the slice's gradient is stored, the entries' parts are there
        auto put = [&](uint32_t e) {
            const int32_t id = sm_id[e];
            if (id < (int32_t)s.lo || id >= (int32_t)s.hi) return;
            float take = sm_x[e];
            if (twice) {   // the first of its id collects the others' parts, in their order
                take = 0.f;
                for (uint32_t o = 0; o < n_entries; ++o)
                    if (sm_id[o] == id) {
                        if (o < e) return;
                        take += sm_x[o];
                    }
            }
            from_f32(out[id], grad(sm_z[e]) - take);
        };
        if (!skip) {
            for (uint32_t e = tid; e < a.k; e += kThreads) put(e);
            if (tid == kThreads - 1) put(a.k);
        }
        if (twice) __syncthreads();   // the next row overwrites entries that others read
    }
    pdl_leave();
}

// ---------------------------------------------------------------------- host

int check(const bf16opt_distill_t *d, const void *loss, bool need_loss, const void *lse, bool need_lse, const float *dloss,
          const void *dlogits, uint64_t dlogits_stride, bool grad) {
    auto bad = [](const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("distill: ") + m); };
    if (!d) return bad("the descriptor is NULL");
    if (!type_ok(d->logits_type) || !type_ok(d->teacher_type)) return bad("unknown element type");
    if (!index_ok(d->ids_type) || !index_ok(d->labels_type)) return bad("unknown index type");
    if (d->vocab < 1 || d->vocab > (1u << 30)) return bad("vocab must lie in [1, 2^30]");
    if (d->k > BF16OPT_DISTILL_MAX_K) return bad("k exceeds BF16OPT_DISTILL_MAX_K");
    if (!(std::isfinite(d->temperature) && d->temperature > 0.f) || !std::isfinite(1.f / d->temperature))
        return bad("temperature must be finite and > 0");
    if (!(std::isfinite(d->kl_weight) && d->kl_weight >= 0.f) || !(std::isfinite(d->ce_weight) && d->ce_weight >= 0.f))
        return bad("kl_weight and ce_weight must be finite and >= 0");
    if (d->logits_stride < d->vocab || (grad && dlogits_stride < d->vocab)) return bad("a row stride is below vocab");
    if (d->k && (d->ids_stride < d->k || d->teacher_stride < d->k)) return bad("a teacher's row stride is below k");
    const uint64_t eb = type_bytes(d->logits_type);
    uint64_t zb = 0, gb = 0, ib = 0, tb = 0;
    if (!span_bytes(d->rows, d->logits_stride, d->vocab, eb, zb) ||
        (grad && !span_bytes(d->rows, dlogits_stride, d->vocab, eb, gb)) ||
        (d->k && (!span_bytes(d->rows, d->ids_stride, d->k, index_bytes(d->ids_type), ib) ||
                  !span_bytes(d->rows, d->teacher_stride, d->k, type_bytes(d->teacher_type), tb))) ||
        d->rows >= (1ull << 40))
        return bad("the sizes overflow");
    if (d->rows == 0) return BF16OPT_OK;
    if (!d->logits || (d->k && (!d->teacher_ids || !d->teacher_logits))) return bad("an input pointer is NULL");
    if ((need_loss && !loss) || (need_lse && !lse) || (grad && !dlogits)) return bad("an output or saved pointer is NULL");
    if (misaligned(d->logits, eb) || misaligned(dlogits, eb) || (d->k && misaligned(d->teacher_ids, index_bytes(d->ids_type))) ||
        (d->k && misaligned(d->teacher_logits, type_bytes(d->teacher_type))) || misaligned(d->teacher_lse, 4) ||
        misaligned(d->labels, index_bytes(d->labels_type)) || misaligned(d->row_weight, 4) || misaligned(loss, 4) ||
        misaligned(lse, 4) || misaligned(dloss, 4))
        return fail(BF16OPT_ERR_ALIGNMENT, "distill: a pointer is not aligned to its element");
    // outputs against inputs and one another
    struct Part { const void *p; uint64_t n; };
    const uint64_t r4 = d->rows * 4;
    const Part in[] = {{d->logits, zb}, {d->teacher_ids, ib}, {d->teacher_logits, tb}, {d->teacher_lse, r4},
                       {d->labels, d->rows * index_bytes(d->labels_type)}, {d->row_weight, r4}, {dloss, r4},
                       {need_lse ? lse : nullptr, 2 * r4}};
    const Part outs[] = {{dlogits, gb}, {need_loss ? loss : nullptr, r4}, {need_lse ? nullptr : lse, 2 * r4}};
    for (int i = 0; i < 3; ++i) {
        for (const Part &x : in) {
            if (i == 0 && x.p == d->logits && x.p == dlogits && dlogits_stride == d->logits_stride) continue;   // in place
            if (overlap(outs[i].p, outs[i].n, x.p, x.n)) return bad("an output overlaps an input");
        }
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return bad("two outputs overlap");
    }
    return BF16OPT_OK;
}

template <int kThreads, class T, bool FORWARD, bool GRAD, int POWER, bool FAR = false>
int launch_k(const Args &a, unsigned cluster, cudaStream_t stream) {
    auto k = k_distill<kThreads, T, FORWARD, GRAD, POWER, FAR>;
    const size_t smem = (size_t)ring_depth(kThreads) * kThreads * kU * 16 + (size_t)(a.k + 1) * 12 + (GRAD ? table_size(a.k) * 4 : 0);
    // As many clusters as fit at once (a cluster of eight cannot use every SM: those of a
    // processing cluster are not a multiple of it), each walking its rows; more would run as a
    // second wave: 57 clusters of eight where 51 fit took 639 us on 2048 rows of 250880 bf16, 51 took 469.
    Launch l{cluster, (unsigned)kThreads, smem, stream, cluster, true};
    int fit = 0;
    const cudaError_t eo = clusters_that_fit(l, k, fit);
    if (eo != cudaSuccess) return fail_cuda(eo, "distill occupancy");
    // in equal shares: 512 rows on 51 clusters would be 11 rows for some, so 47 do
    const uint64_t turns = (a.rows + fit - 1) / fit;
    l.grid = (unsigned)((a.rows + turns - 1) / turns) * cluster;
    const cudaError_t e = launch(l, k, a);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "distill kernel launch");
}

template <class T, bool FORWARD, bool GRAD>
int launch_t(const Args &a, int power, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "distill: no CUDA device");
    // CTAs per row.  With both passes: a slice of at most three rings, so that what is read again is
    // still in L2 (two rings 444 us, three 411 us, six 470 us on 2048 x 250880). The backward pass:
    // slices of at most 8192 vectors, since fewer rows at a time read and write closer together
    // (1024 x 250880: 189 us with a CTA per row, 171 us with four; the forward pass does not care).
    // With few rows: so many that the SMs are used.
    constexpr bool kBoth = FORWARD && GRAD;
    const uint64_t vecs = a.vocab / Vec<T>::N + 1;
    const bool large = kBoth && vecs > kShortRow;
    const uint64_t ring = large ? (uint64_t)ring_depth(kLarge) * kU * kLarge : (uint64_t)ring_depth(kSmall) * kU * kSmall;
    unsigned cluster = 1;
    while (cluster < kMaxCluster && ((kBoth && vecs / cluster > ring * 3) ||
                                     (!FORWARD && vecs / cluster > 8192) ||
                                     (a.rows * cluster <= (uint64_t)sms && vecs / cluster > 4 * kSmall)))
        cluster *= 2;
    auto go = [&](auto p) {
        constexpr int POWER = decltype(p)::value;
        if constexpr (kBoth)
            if (large) return launch_k<kLarge, T, FORWARD, GRAD, POWER>(a, cluster, stream);
        const int rc = launch_k<kSmall, T, FORWARD, GRAD, POWER>(a, cluster, stream);
        if constexpr (!FORWARD)
            if (rc == BF16OPT_OK) return launch_k<kSmall, T, true, true, POWER, true>(a, cluster, stream);
        return rc;
    };
    switch (power) {
    case 0: return go(std::integral_constant<int, 0>());
    case 2: return go(std::integral_constant<int, 2>());
    case 4: return go(std::integral_constant<int, 4>());
    default: return go(std::integral_constant<int, 1>());
    }
}

template <bool FORWARD, bool GRAD>
int run(const bf16opt_distill_t *d, const float *lse_in, const float *dloss, float *loss, float *lse_out, void *dlogits,
        uint64_t dlogits_stride, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    const int rc = check(d, loss, FORWARD, FORWARD ? (const void *)lse_out : lse_in, !FORWARD, dloss, dlogits, dlogits_stride, GRAD);
    if (rc != BF16OPT_OK || d->rows == 0) return rc;
    Args a;
    a.rows = d->rows, a.vocab = d->vocab, a.k = d->kl_weight != 0.f ? d->k : 0;
    a.teacher_type = d->teacher_type, a.ids_type = d->ids_type, a.labels_type = d->labels_type;
    a.logits = d->logits, a.logits_stride = d->logits_stride;
    a.ids = d->teacher_ids, a.ids_stride = d->ids_stride;
    a.teacher = d->teacher_logits, a.teacher_stride = d->teacher_stride, a.teacher_lse = d->teacher_lse;
    a.labels = d->labels, a.row_weight = d->row_weight;
    a.kl_weight = d->kl_weight, a.ce_weight = d->labels ? d->ce_weight : 0.f;
    a.temperature = a.kl_weight != 0.f ? d->temperature : 1.f;   // the label's term alone: everything at 1
    a.inv_t = 1.f / a.temperature;
    a.dloss = dloss, a.lse_in = lse_in, a.loss = loss, a.lse_out = lse_out;
    a.dlogits = dlogits, a.dlogits_stride = dlogits_stride;
    int power = a.ce_weight == 0.f || a.temperature == 1.f ? 0 : 1;
    if (power && (a.temperature == 2.f || a.temperature == 4.f)) power = (int)a.temperature;
    return d->logits_type == BF16OPT_TYPE_BF16 ? launch_t<__nv_bfloat16, FORWARD, GRAD>(a, power, (cudaStream_t)stream)
                                               : launch_t<float, FORWARD, GRAD>(a, power, (cudaStream_t)stream);
}

}  // namespace
}  // namespace bf16ops

extern "C" int bf16opt_distill_forward(const bf16opt_distill_t *d, float *loss, float *lse, void *stream) {
    return bf16ops::guarded([&] { return bf16ops::run<true, false>(d, nullptr, nullptr, loss, lse, nullptr, 0, stream); });
}

extern "C" int bf16opt_distill_backward(const bf16opt_distill_t *d, const float *lse, const float *dloss, void *dlogits,
                                        uint64_t dlogits_stride, void *stream) {
    return bf16ops::guarded(
        [&] { return bf16ops::run<false, true>(d, lse, dloss, nullptr, nullptr, dlogits, dlogits_stride, stream); });
}

extern "C" int bf16opt_distill_loss_grad(const bf16opt_distill_t *d, const float *dloss, float *loss, float *lse,
                                         void *dlogits, uint64_t dlogits_stride, void *stream) {
    return bf16ops::guarded(
        [&] { return bf16ops::run<true, true>(d, nullptr, dloss, loss, lse, dlogits, dlogits_stride, stream); });
}
