// distill.cu -- distillation from a teacher's top logits, forward and backward
// (bf16opt_distill_* of include/bf16opt.h).
//
// A row's loss needs the log-sum-exp of its logits and its gradient needs the
// logits again.  A cluster of CTAs takes a row: each CTA streams its slice of
// the row once, keeping a running maximum and sum per thread, and leaves the
// slice in its shared memory; the CTAs' sums meet through distributed shared
// memory; then each CTA writes its slice's gradient from the copy it kept.  So
// every logit is read from HBM once and every gradient written once, the least
// the operator can do (4 bytes per bf16 logit).
//
// The teacher's k entries of a row (and the label, as one more entry) are held
// in shared memory by every CTA of the cluster.  Their softmax is computed by
// each CTA by itself, and their part of the gradient is put on top of the
// slice's: an entry's element is recomputed and stored again with everything
// that its id collects, rounded once.
#include <cooperative_groups.h>

#include <algorithm>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace bf16ops {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kU = 4;                 // vectors in flight per thread
constexpr int kMaxCluster = 8;
constexpr int kResident = 3;          // CTAs per SM that the registers allow

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
// exp((z - max) / T) and (TWO) exp(z - max).
struct Stat {
    float m, st, s1;
};
// The teacher's: maximum of x = t / T, sum e of exp(x - max), sum of e (x - z / T).
struct Teach {
    float m, s, d;
};

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ Stat join(const Stat &a, const Stat &b, float c_t) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    const float m = safe_max(r.m);
    r.st = a.st * ex2((a.m - m) * c_t) + b.st * ex2((b.m - m) * c_t);
    r.s1 = a.s1 * ex2((a.m - m) * kLog2e) + b.s1 * ex2((b.m - m) * kLog2e);
    return r;
}
__device__ __forceinline__ Teach join(const Teach &a, const Teach &b) {
    Teach r;
    r.m = fmaxf(a.m, b.m);
    const float m = safe_max(r.m);
    const float ea = ex2((a.m - m) * kLog2e), eb = ex2((b.m - m) * kLog2e);
    r.s = a.s * ea + b.s * eb;
    r.d = (ea > 0.f ? a.d * ea : 0.f) + (eb > 0.f ? b.d * eb : 0.f);   // a d of +inf (masked z) may meet a weight of 0
    return r;
}

// A row's slice of one CTA: `head` elements before the first 16-byte boundary
// and `tail` after the last whole vector are the first and the last CTA's.
struct Slice {
    uint32_t head, nv, v0, v1;        // whole row: leading elements, vectors; this CTA's vectors [v0, v1)
    uint32_t tail0, lo, hi;           // first trailing element; this CTA's elements are [lo, hi)
};
template <class T>
__device__ __forceinline__ Slice slice_of(const T *row, uint32_t vocab, uint32_t rank, uint32_t ranks) {
    constexpr uint32_t N = Vec<T>::N;
    Slice s;
    const uint32_t off = (uint32_t)((uintptr_t)row & 15u) / (uint32_t)sizeof(T);
    s.head = off ? N - off : 0u;
    if (s.head > vocab) s.head = vocab;
    s.nv = (vocab - s.head) / N;
    s.tail0 = s.head + s.nv * N;
    s.v0 = (uint32_t)((uint64_t)s.nv * rank / ranks);
    s.v1 = (uint32_t)((uint64_t)s.nv * (rank + 1) / ranks);
    s.lo = rank == 0 ? 0u : s.head + s.v0 * N;
    s.hi = rank + 1 == ranks ? vocab : s.head + s.v1 * N;
    return s;
}

// Stores one vector of the gradient: whole where the output row's vectors are
// aligned as the input row's, else element by element.
template <class T>
__device__ __forceinline__ void store_vec(T *out, const float (&g)[Vec<T>::N], bool whole) {
    const uint4 v = Vec<T>::pack(g);
    if (whole) {
        __stcs(reinterpret_cast<uint4 *>(out), v);
    } else {
        const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) out[i] = e[i];
    }
}

// FORWARD: the row's sums are computed here (else read from lse_in).  GRAD: the
// gradient is written.  TWO: the sum and the gradient at temperature 1 are
// needed next to those at T.  KEEP: the slice stays in shared memory between
// the two (else it is read again).
template <class T, bool FORWARD, bool GRAD, bool TWO, bool KEEP>
__global__ void __launch_bounds__(kThreads, kResident) k_distill(const Args a, uint32_t slice_vecs) {
    constexpr int N = Vec<T>::N;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    // slice | ids, x (then what the entry takes off the gradient), z of the entries
    uint4 *keep = reinterpret_cast<uint4 *>(smem_raw);
    int32_t *sm_id = reinterpret_cast<int32_t *>(smem_raw + (KEEP ? (size_t)slice_vecs * 16 : 0));
    float *sm_x = reinterpret_cast<float *>(sm_id + (a.k + 1));
    float *sm_z = sm_x + (a.k + 1);
    __shared__ Stat sm_stat[kWarps];
    __shared__ Teach sm_teach[kWarps];
    __shared__ Stat sm_cluster[2][kMaxCluster];

    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t n_entries = a.k + 1;   // the label is the last one
    const float c_t = a.inv_t * kLog2e;
    pdl_enter();
    if (FORWARD && ranks > 1) cluster.sync();   // every CTA's shared memory exists

    uint32_t turn = 0;
    for (uint64_t row = blockIdx.x / ranks; row < a.rows; row += gridDim.x / ranks) {
        const T *z = reinterpret_cast<const T *>(a.logits) + row * a.logits_stride;
        T *out = GRAD ? reinterpret_cast<T *>(a.dlogits) + row * a.dlogits_stride : nullptr;
        const Slice s = slice_of(z, a.vocab, rank, ranks);
        const bool whole = GRAD && (((uintptr_t)out ^ (uintptr_t)z) & 15u) == 0;
        const uint4 *zv = reinterpret_cast<const uint4 *>(z + s.head);
        const float w = a.row_weight ? a.row_weight[row] : 1.f;

        if (w == 0.f) {   // not read: zeros
            if (GRAD) {
                float zero[N] = {};
                for (uint32_t v = s.v0 + tid; v < s.v1; v += kThreads) store_vec<T>(out + s.head + (size_t)v * N, zero, whole);
                if (rank == 0 && tid < s.head) from_f32(out[tid], 0.f);
                if (rank + 1 == ranks && tid < a.vocab - s.tail0) from_f32(out[s.tail0 + tid], 0.f);
            }
            if (FORWARD && rank == 0 && tid == 0) {
                a.loss[row] = 0.f;
                if (a.lse_out) a.lse_out[2 * row] = a.lse_out[2 * row + 1] = 0.f;
            }
            continue;
        }

        // ---- the teacher's entries and the label
        Teach te = {-INFINITY, 0.f, 0.f};
        for (uint32_t e = tid; e < a.k; e += kThreads) {
            const int64_t id64 = load_index(a.ids, a.ids_type, row * a.ids_stride + e);
            const float x = load_typed(a.teacher, a.teacher_type, row * a.teacher_stride + e) * a.inv_t;
            const bool there = id64 >= 0 && id64 < (int64_t)a.vocab && x != -INFINITY;
            const int32_t id = there ? (int32_t)id64 : -1;
            const float zi = there ? to_f32(z[id]) : 0.f;
            sm_id[e] = id, sm_x[e] = x, sm_z[e] = zi;
            if (there) {
                const Teach one = {x, 1.f, x - zi * a.inv_t};
                te = join(te, one);
            }
        }
        if (tid == 0) {
            int64_t id64 = -1;
            if (a.ce_weight != 0.f) id64 = load_index(a.labels, a.labels_type, row);
            const bool there = id64 >= 0 && id64 < (int64_t)a.vocab;
            sm_id[a.k] = there ? (int32_t)id64 : -1;
            sm_z[a.k] = there ? to_f32(z[id64]) : 0.f;
        }

        // ---- the slice's running maximum and sums
        Stat st = {-INFINITY, 0.f, 0.f};
        if (FORWARD) {
            for (uint32_t v = s.v0 + tid; v < s.v1; v += kThreads * kU) {
                uint4 q[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const uint32_t j = v + u * kThreads;
                    if (j < s.v1) q[u] = KEEP || !GRAD ? __ldcs(zv + j) : __ldcg(zv + j);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const uint32_t j = v + u * kThreads;
                    if (j >= s.v1) break;
                    if (KEEP) keep[j - s.v0] = q[u];
                    float f[N];
                    Vec<T>::unpack(q[u], f);
                    float mx = f[0];
#pragma unroll
                    for (int i = 1; i < N; ++i) mx = fmaxf(mx, f[i]);
                    if (mx > st.m) {
                        st.st *= ex2((st.m - mx) * c_t);
                        if (TWO) st.s1 *= ex2((st.m - mx) * kLog2e);
                        st.m = mx;
                    }
                    const float m = safe_max(st.m);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        st.st += ex2((f[i] - m) * c_t);
                        if (TWO) st.s1 += ex2((f[i] - m) * kLog2e);
                    }
                }
            }
            uint32_t at = 0xffffffffu;
            if (rank == 0 && tid < s.head) at = tid;
            else if (rank + 1 == ranks && tid >= 32 && tid - 32 < a.vocab - s.tail0) at = s.tail0 + tid - 32;
            if (at != 0xffffffffu) {
                const float f = to_f32(z[at]);
                const float one = f == -INFINITY ? 0.f : f == f ? 1.f : f;   // a NaN stays one
                st = join(st, Stat{f == f ? f : -INFINITY, one, one}, c_t);
            }
        }

        // ---- joined over the CTA and the cluster, in a fixed order
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (FORWARD) {
                Stat b;
                b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
                b.st = __shfl_xor_sync(0xffffffffu, st.st, o);
                b.s1 = TWO ? __shfl_xor_sync(0xffffffffu, st.s1, o) : 0.f;
                st = join(st, b, c_t);
            }
            Teach t;
            t.m = __shfl_xor_sync(0xffffffffu, te.m, o);
            t.s = __shfl_xor_sync(0xffffffffu, te.s, o);
            t.d = __shfl_xor_sync(0xffffffffu, te.d, o);
            te = join(te, t);
        }
        if (lane == 0) {
            sm_stat[warp] = st;
            sm_teach[warp] = te;
        }
        __syncthreads();
        te = sm_teach[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) te = join(te, sm_teach[i]);
        float lse_t, lse_1;
        bool empty;   // no logit but -inf in the row
        // q = exp2((z - base_t) c_t + rest_t): the base near the row's top, so that z - base is exact there
        float base_t, rest_t, base_1, rest_1;
        if (FORWARD) {
            st = sm_stat[0];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) st = join(st, sm_stat[i], c_t);
            if (ranks > 1) {
                if (tid < ranks) *cluster.map_shared_rank(&sm_cluster[turn & 1][rank], tid) = st;
                cluster.sync();
                st = sm_cluster[turn & 1][0];
                for (uint32_t i = 1; i < ranks; ++i) st = join(st, sm_cluster[turn & 1][i], c_t);
                ++turn;
            }
            const float m = safe_max(st.m);
            empty = st.m == -INFINITY && st.st == 0.f;
            lse_t = empty ? -INFINITY : m * a.inv_t + logf(st.st);
            lse_1 = empty ? -INFINITY : (TWO ? m + logf(st.s1) : lse_t);
            base_t = base_1 = m;
            rest_t = empty ? 0.f : -log2f(st.st);
            rest_1 = TWO && !empty ? -log2f(st.s1) : 0.f;
        } else {
            lse_t = a.lse_in[2 * row];
            lse_1 = a.lse_in[2 * row + 1];
            empty = lse_t == -INFINITY;
            base_t = empty ? 0.f : lse_t * a.temperature;
            rest_t = empty ? 0.f : fmaf(lse_t, a.temperature, -base_t) * -c_t;
            base_1 = empty ? 0.f : lse_1;
            rest_1 = 0.f;
        }

        // ---- the row's loss
        const bool some = te.s != 0.f;   // the teacher has entries here (NaN counts)
        const float lse_teacher = a.teacher_lse ? a.teacher_lse[row] : te.m + logf(te.s);
        const float mass = !some ? 0.f : a.teacher_lse ? te.s * ex2((te.m - lse_teacher) * kLog2e) : te.s == te.s ? 1.f : te.s;
        const bool has_label = sm_id[a.k] >= 0;
        if (FORWARD && rank == 0 && tid == 0) {
            float kl = 0.f, ce = 0.f;
            if (some && a.kl_weight != 0.f && mass != 0.f)
                kl = empty ? INFINITY : a.kl_weight * a.temperature * a.temperature * mass * (te.d / te.s + (lse_t - lse_teacher));
            if (has_label) ce = empty ? INFINITY : a.ce_weight * (lse_1 - sm_z[a.k]);
            a.loss[row] = w * (kl + ce);
            if (a.lse_out) a.lse_out[2 * row] = lse_t, a.lse_out[2 * row + 1] = lse_1;
        }
        if (!GRAD) {
            __syncthreads();
            continue;
        }

        // ---- the gradient of the slice
        const float up = w * (a.dloss ? a.dloss[row] : 1.f);
        const float hard = has_label ? up * a.ce_weight : 0.f;
        const float soft = up * a.kl_weight * a.temperature;
        float a_t = soft * mass, a_1 = hard;
        if (!TWO) a_t += hard, a_1 = 0.f;   // both terms have the same softmax
        auto grad = [&](float f) {
            float g = a_t * ex2(fmaf(f - base_t, c_t, rest_t));
            if (TWO) g = fmaf(a_1, ex2(fmaf(f - base_1, kLog2e, rest_1)), g);
            return g;
        };
        for (uint32_t v = s.v0 + tid; v < s.v1; v += kThreads * kU) {
            uint4 q[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const uint32_t j = v + u * kThreads;
                if (j < s.v1) q[u] = KEEP ? keep[j - s.v0] : __ldcs(zv + j);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const uint32_t j = v + u * kThreads;
                if (j >= s.v1) break;
                float f[N];
                Vec<T>::unpack(q[u], f);
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = grad(f[i]);
                store_vec<T>(out + s.head + (size_t)j * N, f, whole);
            }
        }
        if (rank == 0 && tid < s.head) from_f32(out[tid], grad(to_f32(z[tid])));
        if (rank + 1 == ranks && tid < a.vocab - s.tail0)
            from_f32(out[s.tail0 + tid], grad(to_f32(z[s.tail0 + tid])));

        // ---- the entries of the slice
        for (uint32_t e = tid; e < a.k; e += kThreads) sm_x[e] = soft * ex2((sm_x[e] - lse_teacher) * kLog2e);
        if (tid == 0) sm_x[a.k] = hard;
        __syncthreads();   // the slice's gradient is stored, the entries' parts are there
        for (uint32_t e = tid; e < n_entries; e += kThreads) {
            const int32_t id = sm_id[e];
            if (id < (int32_t)s.lo || id >= (int32_t)s.hi) continue;
            bool first = true;
            float take = 0.f;
            for (uint32_t o = 0; o < n_entries; ++o)
                if (sm_id[o] == id) {
                    if (o < e) first = false;
                    take += sm_x[o];
                }
            if (first) from_f32(out[id], grad(sm_z[e]) - take);
        }
        __syncthreads();   // the next row overwrites the entries
    }
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

// Shared memory that a slice may take: three CTAs of an SM's 227 KB where the
// cluster can be made large enough for that, else one.
constexpr size_t kSliceMany = 64 * 1024, kSliceOne = 200 * 1024;

template <class T, bool FORWARD, bool GRAD, bool TWO, bool KEEP>
int launch_k(const Args &a, unsigned cluster, uint32_t slice_vecs, int sms, cudaStream_t stream) {
    auto k = k_distill<T, FORWARD, GRAD, TWO, KEEP>;
    const size_t smem = (KEEP ? (size_t)slice_vecs * 16 : 0) + (size_t)(a.k + 1) * 12;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return fail_cuda(e, "distill kernel attribute");
    }
    // enough clusters for the CTAs that an SM can hold; each walks its rows
    const uint64_t per_sm = std::min<uint64_t>(kResident, (227 * 1024) / (smem + 2048));
    const uint64_t clusters = std::min<uint64_t>(a.rows, std::max<uint64_t>(1, (uint64_t)sms * per_sm / cluster));
    Launch l{(unsigned)(clusters * cluster), (unsigned)kThreads, smem, stream, cluster, true};
    const cudaError_t e = launch(l, k, a, slice_vecs);
    return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "distill kernel launch");
}

template <class T, bool FORWARD, bool GRAD>
int launch_t(const Args &a, bool two, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "distill: no CUDA device");
    // CTAs per row: enough that a slice leaves room for three CTAs per SM, and,
    // with few rows, enough that the SMs are used.
    const uint64_t vecs = a.vocab / Vec<T>::N + 1;
    unsigned cluster = 1;
    while (cluster < kMaxCluster && ((vecs * 16 + cluster - 1) / cluster > kSliceMany ||
                                     (a.rows * cluster * 2 <= (uint64_t)sms && vecs / cluster > 4 * kThreads)))
        cluster *= 2;
    const uint32_t slice_vecs = (uint32_t)(vecs / cluster + 1);
    const bool keep = FORWARD && GRAD && (size_t)slice_vecs * 16 <= kSliceOne;
    if constexpr (FORWARD && GRAD) {
        if (keep)
            return two ? launch_k<T, FORWARD, GRAD, true, true>(a, cluster, slice_vecs, sms, stream)
                       : launch_k<T, FORWARD, GRAD, false, true>(a, cluster, slice_vecs, sms, stream);
    }
    return two ? launch_k<T, FORWARD, GRAD, true, false>(a, cluster, slice_vecs, sms, stream)
               : launch_k<T, FORWARD, GRAD, false, false>(a, cluster, slice_vecs, sms, stream);
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
    const bool two = a.ce_weight != 0.f && a.temperature != 1.f;
    return d->logits_type == BF16OPT_TYPE_BF16 ? launch_t<__nv_bfloat16, FORWARD, GRAD>(a, two, (cudaStream_t)stream)
                                               : launch_t<float, FORWARD, GRAD>(a, two, (cudaStream_t)stream);
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
