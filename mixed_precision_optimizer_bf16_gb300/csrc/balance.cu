// balance.cu -- a router's choice of experts, their counts, the balance loss and
// the z-loss, forward and backward (bf16opt_balance_* of include/bf16opt.h).
//
// A warp takes a token: each lane holds a run of PER experts in registers, so
// the softmax, the k largest logits and the mean probabilities come from one
// read of the logits.  A CTA walks a contiguous run of tokens and keeps the
// sums of the group it is in; a group that lies within one CTA is finished
// there, the others leave partial sums that a second kernel joins in the CTAs'
// order.  (f_e, the share of tokens of an expert, is known only after the last
// token, so the gradient is a second pass.)
//
// Measured on one GB300: 262144 tokens, 256 experts, 8 of them, bf16: forward 121 us, 1.1 TB/s, join 10 us,
// backward 68 us, 4.2 TB/s; both ways 198 us in a row.  The forward pass is bound by integer instructions (69 %
// of that pipe's cycles, 76 % of the issue slots): 430 a token, most of them the choice's.  The backward pass is
// bound by issue (70 % of the slots) and a token's sums and lookups in shared memory.  16384 tokens of 64 FP32
// experts in 8 groups: 13 + 6 + 7 us, which the host's calls take longer than.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace bf16ops {
namespace {

// CTAs of an SM in the backward pass, by the experts of a lane: three have 85 registers a thread (at 64 that of 256
// experts spills: 262144 x 256 took 266 us both ways, 220 us so; 131072 x 256 FP32 backward 145 against 52 us); up to
// 64 experts 64 registers are enough (262144 x 64 backward: FP32 52 against 64 us, bf16 62 against 80 us).
__host__ __device__ constexpr int back_resident(int per) { return per <= 2 ? 4 : per <= 8 ? 3 : 1; }
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Args {
    uint64_t tokens, groups, per_group;
    uint32_t experts, k;
    int renormalise;
    const void *logits;
    uint64_t stride;
    bool vec;                       // every lane's run is one aligned run of the row
    const uint8_t *mask;
    float balance_weight, z_weight;
    int32_t *ids;
    float *weights;
    int32_t *counts;
    float *loss, *lse, *live;       // live: tokens of each group that count
    // scratch: losses [groups]; then per CTA two slots of experts sums, experts counts, squares, live
    float *group_loss, *slots;
    uint32_t teams;
};

__host__ __device__ inline size_t slot_floats(uint32_t experts) { return 2 * (size_t)experts + 2; }

// Logits as unsigned keys in their order: -inf (an expert that is off) 0, NaN 1,
// then the numbers; both zeros are one key.
__device__ __forceinline__ uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z + 0.f);
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return z != z ? 1u : z == -INFINITY ? 0u : k;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    if (k == 1u) return NAN;
    if (k == 0u) return -INFINITY;
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A token's choice, one largest logit after another, is by far the most of the
// forward pass's work.  For bf16 logits a key holds the logit's 16 bits in their order
// and, below them, the expert counted backwards, so that keys are distinct and the
// lowest expert wins a tie: a lane sorts its keys once (a network of exchanges), and a
// choice is one reduction over the lanes' largest and one step of the winner's list.
// FP32 logits leave no room for the expert: there a choice is a reduction and a
// ballot; a lane of up to 8 experts keeps its keys sorted beside their experts (262144
// tokens forward, 64 experts 120 us, 128 experts 175 us), a longer one searches its run again when
// it has won (so throughout: 133 and 207 us).  Under kOff16 come experts that are off.
constexpr uint32_t kOff16 = 0x00800000u;

// Eight keys in descending order: an odd-even merge network of 19 exchanges.
__device__ __forceinline__ void order(uint32_t &a, uint32_t &b) {
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi, b = lo;
}
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
    // odd-even merge sort (Batcher): p runs over the merged lengths, q over the exchange distances
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order(k[i + j], k[i + j + q]);
}

// A lane's run of a row as it lies in memory: experts [lane * PER, lane * PER + PER), -inf beyond.
template <class T, int PER>
struct RunOf {
    static constexpr int W = PER * (int)sizeof(T) < 4 ? 1 : PER * (int)sizeof(T) / 4;
    uint32_t w[W];
};
template <class T, int PER>
__device__ __forceinline__ RunOf<T, PER> load_run(const T *row, uint32_t experts, uint32_t lane, bool vec) {
    RunOf<T, PER> r;
    constexpr int W = RunOf<T, PER>::W;
    const uint32_t e0 = lane * PER;
    if (vec && PER * sizeof(T) >= 4) {
        if (e0 < experts) {
            if constexpr (W >= 4) {
#pragma unroll
                for (int i = 0; i < W / 4; ++i) {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + e0) + i);
                    r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
                }
            } else if constexpr (W == 2) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(row + e0));
                r.w[0] = v.x, r.w[1] = v.y;
            } else if constexpr (PER * sizeof(T) == 4) {
                r.w[0] = __ldcs(reinterpret_cast<const uint32_t *>(row + e0));
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) r.w[i] = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        }
        return r;
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < PER; ++i) r.w[i] = e0 + i < experts ? __float_as_uint(to_f32(row[e0 + i])) : 0xff800000u;
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t lo = 0xff80u, hi = 0xff80u;
            if (e0 + 2 * i < experts) lo = __bfloat16_as_ushort(row[e0 + 2 * i]);
            if (PER > 1 && e0 + 2 * i + 1 < experts) hi = __bfloat16_as_ushort(row[e0 + 2 * i + 1]);
            r.w[i] = lo | hi << 16;
        }
    }
    return r;
}
template <class T, int PER>
__device__ __forceinline__ void unpack_run(const RunOf<T, PER> &r, float (&z)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if constexpr (sizeof(T) == 4) z[i] = __uint_as_float(r.w[i]);
        else z[i] = i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
    }
}
template <class T, int PER>
__device__ __forceinline__ void store_run(T *row, uint32_t experts, uint32_t lane, bool vec, const float (&g)[PER]) {
    const uint32_t e0 = lane * PER;
    constexpr int BYTES = PER * (int)sizeof(T);
    if (vec && BYTES >= 16) {
        if constexpr (BYTES >= 16) {
            constexpr int N = Vec<T>::N;
            if (e0 < experts) {
#pragma unroll
                for (int v = 0; v < PER / N; ++v) {
                    float f[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) f[i] = g[v * N + i];
                    reinterpret_cast<uint4 *>(row + e0)[v] = Vec<T>::pack(f);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (e0 + i < experts) from_f32(row[e0 + i], g[i]);
}

__device__ __forceinline__ float reciprocal(float x) {   // to one unit in the last place
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The z-loss of a group; 0 where its weight is, though a square of far logits does not fit FP32.
__device__ __forceinline__ float z_loss(float weight, float squares, float n) { return weight * ((weight != 0.f ? squares : 0.f) / n); }
// sum over the CTA, the same bits in every thread
__device__ __forceinline__ float cta_sum(float v, float *buf) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kWarps; ++i) s += buf[i];
    return s;
}

template <class T, int PER>
__global__ void __launch_bounds__(kThreads, PER <= 8 ? 4 : 1) k_balance_forward(const Args a) {
    constexpr bool kPacked = sizeof(T) == 2 && PER >= 2 && PER <= 8;   // keys of 16 bits and the expert
    extern __shared__ float sm[];
    float *sm_p = sm;                                             // [warps][experts]
    int *sm_count = reinterpret_cast<int *>(sm + kWarps * a.experts);   // [experts]
    __shared__ float sm_sq[kWarps], sm_buf[kWarps];
    __shared__ int sm_live[kWarps];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = blockIdx.x;
    pdl_enter();
    const uint64_t t0 = team_row(a.tokens, a.teams, team), t1 = team_row(a.tokens, a.teams, team + 1);
    const T *logits = reinterpret_cast<const T *>(a.logits);
    float whole = 0.f;   // one CTA: the loss of all groups
    for (uint64_t g = t0 / a.per_group; g * a.per_group < t1; ++g) {
        const uint64_t first = g * a.per_group, last = first + a.per_group;
        const uint64_t b = first > t0 ? first : t0, e = last < t1 ? last : t1;
        for (uint32_t i = threadIdx.x; i < a.experts; i += kThreads) sm_count[i] = 0;
        __syncthreads();
        float sum[PER] = {};
        float squares = 0.f;
        int live = 0;
        // a token's logits are asked for while the two before are worked on
        RunOf<T, PER> ahead, after;
        uint8_t on_ahead = 0, on_after = 0;
        uint64_t t = b + warp;
        uint32_t todo = t < e ? (uint32_t)((e - t + kWarps - 1) / kWarps) : 0u, to_fetch = todo;   // tokens of this warp
        const T *row = logits + t * a.stride;
        const uint8_t *mask = a.mask ? a.mask + t : nullptr;
        auto fetch = [&]() {
            ahead = after, on_ahead = on_after;
            if (to_fetch == 0) return;
            --to_fetch;
            on_after = mask ? *mask : 1;
            after = load_run<T, PER>(row, a.experts, lane, a.vec);
            row += kWarps * a.stride;
            if (mask) mask += kWarps;
        };
        fetch();
        fetch();
        float *lse_to = a.lse + t, *weight_to = a.weights + t * a.k + lane;
        int32_t *id_to = a.ids + t * a.k + lane;
        for (; todo != 0; --todo, lse_to += kWarps, weight_to += kWarps * a.k, id_to += kWarps * a.k) {
            const RunOf<T, PER> run = ahead;
            const bool on = on_ahead != 0;
            fetch();
            float lse = -INFINITY;
            int32_t my_id = -1;     // lane c keeps choice c
            float my_p = 0.f;
            if (on) {
                float z[PER];
                unpack_run<T, PER>(run, z);
                float mx = z[0];
#pragma unroll
                for (int i = 1; i < PER; ++i) mx = fmaxf(mx, z[i]);
                mx = warp_max(mx);      // NaN passed over
                const float m = mx == -INFINITY ? 0.f : mx;
                float p[PER], s;
                if constexpr (PER == 1) {
                    s = p[0] = ex2((z[0] - m) * kLog2e);
                } else {
                    float2 s2 = both(0.f);
#pragma unroll
                    for (int i = 0; i < PER; i += 2) {
                        const float2 d = mul2(add2(make_float2(z[i], z[i + 1]), both(-m)), both(kLog2e));
                        p[i] = ex2(d.x), p[i + 1] = ex2(d.y);
                        s2 = add2(s2, make_float2(p[i], p[i + 1]));
                    }
                    s = s2.x + s2.y;
                }
                s = warp_sum(s);
                if (s != 0.f) {         // some expert is there
                    const float inv = reciprocal(s);
                    lse = m + logf(s);
#pragma unroll
                    for (int i = 0; i < PER; ++i) sum[i] = fmaf(p[i], inv, sum[i]);
                    squares = fmaf(lse, lse, squares);
                    ++live;
                    const bool odd = s != s;   // a NaN is among them: it comes after every number
                    if constexpr (kPacked) {
                        uint32_t key[PER], mine = 0, least = kOff16;
                        const uint32_t back = 0xffffu - lane * PER;
#pragma unroll
                        for (int i = 0; i < PER / 2; ++i) {   // two logits of a word at once
                            uint32_t w;
                            asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(run.w[i]), "r"(0u));   // both zeros are one
                            w ^= 0x80008000u | (w >> 15 & 0x00010001u) * 0x7fffu;   // ascending as unsigned numbers
                            key[2 * i] = w << 16 | (back - 2 * i), key[2 * i + 1] = (w & 0xffff0000u) | (back - 2 * i - 1);
                        }
                        if (odd) {
                            least = 0x10000u;
#pragma unroll
                            for (int i = 0; i < PER; ++i) {
                                if (z[i] != z[i]) key[i] = (kOff16 - 0x10000u) | (back - i);
                                if (z[i] == -INFINITY) key[i] = 0u;
                            }
                        }
                        sort_keys<PER>(key);
                        auto choose = [&](uint32_t c, int depth) {   // only `depth` keys of a lane can still come
                            const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
                            if (lane == c) mine = top;
                            if (key[0] == top) {
#pragma unroll
                                for (int i = 0; i + 1 < PER; ++i)
                                    if (i < depth) key[i] = key[i + 1];
                                if (depth >= PER) key[PER - 1] = 0u;
                            }
                        };
                        if (a.k <= 8) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (c < (int)a.k) choose(c, 8 - c);
                        } else {
                            for (uint32_t c = 0; c < a.k; ++c) choose(c, PER);
                        }
                        if (mine >= least) {
                            my_id = (int32_t)(0xffffu - (mine & 0xffffu));
                            const uint32_t up = mine & 0xffff0000u;   // the logit back from its key
                            const float my_z = up < kOff16 ? NAN : __uint_as_float(up & 0x80000000u ? up ^ 0x80000000u : ~up & 0xffff0000u);
                            my_p = ex2((my_z - m) * kLog2e) * inv;
                        }
                    } else if constexpr (PER <= 8) {
                        // the lane's keys in descending order, equal ones by their expert: neighbours change places
                        uint32_t key[PER], at[PER];
#pragma unroll
                        for (int i = 0; i < PER; ++i) key[i] = key_of(z[i]), at[i] = lane * PER + i;
#pragma unroll
                        for (int n = PER - 1; n > 0; --n)
#pragma unroll
                            for (int i = 0; i < n; ++i) {
                                const bool swap = key[i + 1] > key[i];
                                const uint32_t k0 = key[i], a0 = at[i];
                                key[i] = swap ? key[i + 1] : k0, key[i + 1] = swap ? k0 : key[i + 1];
                                at[i] = swap ? at[i + 1] : a0, at[i + 1] = swap ? a0 : at[i + 1];
                            }
                        for (uint32_t c = 0; c < a.k; ++c) {
                            const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
                            if (top == 0u) break;
                            const uint32_t from = __ffs(__ballot_sync(0xffffffffu, key[0] == top)) - 1;
                            const int32_t id = (int32_t)__shfl_sync(0xffffffffu, at[0], from);
                            if (lane == c) my_id = id, my_p = ex2((value_of(top) - m) * kLog2e) * inv;
                            const bool won = lane == from;
#pragma unroll
                            for (int i = 0; i + 1 < PER; ++i) key[i] = won ? key[i + 1] : key[i], at[i] = won ? at[i + 1] : at[i];
                            key[PER - 1] = won ? 0u : key[PER - 1];
                        }
                    } else {
                        uint32_t key[PER], best = 0, at = 0;
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            key[i] = key_of(z[i]);
                            if (key[i] > best) best = key[i], at = i;
                        }
                        for (uint32_t c = 0; c < a.k; ++c) {
                            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
                            if (top == 0u) break;
                            const uint32_t from = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
                            const int32_t id = (int32_t)__shfl_sync(0xffffffffu, lane * PER + at, from);
                            if (lane == c) my_id = id, my_p = ex2((value_of(top) - m) * kLog2e) * inv;
                            if (lane == from) {
                                best = 0;
                                uint32_t next = 0;
#pragma unroll
                                for (int i = 0; i < PER; ++i) {
                                    if (i == (int)at) key[i] = 0u;
                                    if (key[i] > best) best = key[i], next = i;
                                }
                                at = next;
                            }
                        }
                    }
                    if (my_id >= 0) atomicAdd(&sm_count[my_id], 1);   // whole numbers: the order does not matter
                    if (a.renormalise) my_p *= reciprocal(warp_sum(my_p));
                }
            }
            if (lane == 0) *lse_to = lse;
            if (lane < a.k) *id_to = my_id, *weight_to = my_id < 0 ? 0.f : my_p;
        }
        // the warps' sums, joined in their order
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane * PER + i < a.experts) sm_p[warp * a.experts + lane * PER + i] = sum[i];
        if (lane == 0) sm_sq[warp] = squares, sm_live[warp] = live;
        __syncthreads();
        float sq = 0.f;
        int n = 0;
        for (int i = 0; i < kWarps; ++i) sq += sm_sq[i], n += sm_live[i];
        if (b == first && e == last) {   // the whole group
            float fp = 0.f;
            for (uint32_t i = threadIdx.x; i < a.experts; i += kThreads) {
                float p = 0.f;
                for (int w = 0; w < kWarps; ++w) p += sm_p[w * a.experts + i];
                a.counts[g * a.experts + i] = sm_count[i];
                fp = fmaf((float)sm_count[i], p, fp);
            }
            fp = cta_sum(fp, sm_buf);
            const float nf = (float)n;
            const float l = n == 0 ? 0.f
                                   : a.balance_weight * (fp / nf) * ((float)a.experts / ((float)a.k * nf)) + z_loss(a.z_weight, sq, nf);
            whole += l;
            if (threadIdx.x == 0) {
                a.live[g] = nf;
                if (a.teams > 1) a.group_loss[g] = l;
            }
        } else {
            float *slot = a.slots + (2 * (size_t)team + (b == first && first > t0 ? 1 : 0)) * slot_floats(a.experts);
            for (uint32_t i = threadIdx.x; i < a.experts; i += kThreads) {
                float p = 0.f;
                for (int w = 0; w < kWarps; ++w) p += sm_p[w * a.experts + i];
                slot[i] = p;
                slot[a.experts + i] = __int_as_float(sm_count[i]);
            }
            if (threadIdx.x == 0) slot[2 * a.experts] = sq, slot[2 * a.experts + 1] = __int_as_float(n);
        }
        __syncthreads();
    }
    if (a.teams == 1 && threadIdx.x == 0) *a.loss = whole / (float)a.groups;
}

// Joins the partial sums of the groups that several CTAs worked on.  WHOLE: one
// cluster for everything, the loss too: a CTA takes a share of the experts
// of one group, or whole groups; the terms meet in rank 0.  Else a CTA per group, and
// k_balance_sum after it.
constexpr int kJoinWarps = 32;
template <bool WHOLE>
__global__ void __launch_bounds__(32 * kJoinWarps) k_balance_join(const Args a) {
    __shared__ float sm_p[kJoinWarps][32];
    __shared__ int sm_c[kJoinWarps][32];
    __shared__ float sm_buf[kJoinWarps], sm_rank[8];
    __shared__ int sm_n[kJoinWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = WHOLE ? cluster.num_blocks() : 1, rank = WHOLE ? cluster.block_rank() : 0;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto cta_total = [&](float v) {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) sm_buf[warp] = v;
        __syncthreads();
        return warp_sum(sm_buf[lane]);   // kJoinWarps is the warp's size
    };
    pdl_enter();
    if (WHOLE && ranks > 1) cluster.sync();
    const size_t sf = slot_floats(a.experts);
    const bool split = WHOLE && a.groups == 1;   // the one group's experts over the CTAs
    float whole = 0.f;
    const uint64_t g0 = split ? 0 : WHOLE ? rank : blockIdx.x, gs = split ? 1 : WHOLE ? ranks : gridDim.x;
    for (uint64_t g = g0; g < a.groups; g += gs) {
        const uint64_t first = g * a.per_group, last = first + a.per_group - 1;
        const uint32_t p0 = team_of(a.tokens, a.teams, first), p1 = team_of(a.tokens, a.teams, last);
        if (p0 == p1) {
            if (WHOLE) whole += a.group_loss[g];
            continue;
        }
        const uint32_t parts = p1 - p0 + 1;
        const uint32_t second = first > team_row(a.tokens, a.teams, p0) ? 1 : 0;
        auto slot = [&](uint32_t i) { return a.slots + (2 * (size_t)(p0 + i) + (i == 0 ? second : 0)) * sf; };
        float sq = 0.f;
        int n = 0;
        for (uint32_t i = threadIdx.x; i < parts; i += 32 * kJoinWarps) {
            const float *s = slot(i);
            sq += s[2 * a.experts];
            n += __float_as_int(s[2 * a.experts + 1]);
        }
        sq = cta_total(sq);
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) sm_n[warp] = n;
        __syncthreads();
        n = __reduce_add_sync(0xffffffffu, sm_n[lane]);
        // experts by 32, the parts by runs over the warps
        float fp = 0.f;
        for (uint32_t c = split ? rank * 32 : 0; c < a.experts; c += (split ? ranks : 1) * 32) {
            const uint32_t e = c + lane;
            float p = 0.f;
            int cnt = 0;
            const uint32_t i0 = parts * warp / kJoinWarps, i1 = parts * (warp + 1) / kJoinWarps;
            if (e < a.experts)
#pragma unroll 8
                for (uint32_t i = i0; i < i1; ++i) {
                    const float *s = slot(i);
                    p += s[e];
                    cnt += __float_as_int(s[a.experts + e]);
                }
            sm_p[warp][lane] = p, sm_c[warp][lane] = cnt;
            __syncthreads();
            if (warp == 0 && e < a.experts) {
                for (int w = 1; w < kJoinWarps; ++w) p += sm_p[w][lane], cnt += sm_c[w][lane];
                a.counts[g * a.experts + e] = cnt;
                fp = fmaf((float)cnt, p, fp);
            }
            __syncthreads();
        }
        fp = cta_total(fp);
        const float nf = (float)n, share = (float)a.experts / ((float)a.k * nf);
        float l = n == 0 ? 0.f : a.balance_weight * (fp / nf) * share;
        if (!split || rank == 0) l += n == 0 ? 0.f : z_loss(a.z_weight, sq, nf);
        if ((!split || rank == 0) && threadIdx.x == 0) {
            a.live[g] = nf;
            if (!WHOLE) a.group_loss[g] = l;
        }
        whole += l;
    }
    if (WHOLE) {
        if (ranks > 1) {
            if (threadIdx.x == 0) *cluster.map_shared_rank(&sm_rank[rank], 0) = whole;
            cluster.sync();
            whole = 0.f;
            if (rank == 0)
                for (uint32_t i = 0; i < ranks; ++i) whole += sm_rank[i];
        }
        if (rank == 0 && threadIdx.x == 0) *a.loss = whole / (float)a.groups;
    }
    pdl_leave();
}

// The groups' losses, summed in order by one CTA.
__global__ void __launch_bounds__(kThreads) k_balance_sum(const float *group_loss, uint64_t groups, float *loss) {
    __shared__ float buf[kWarps];
    pdl_enter();
    float s = 0.f;
    for (uint64_t i = threadIdx.x; i < groups; i += kThreads) s += group_loss[i];
    s = cta_sum(s, buf);
    if (threadIdx.x == 0) *loss = s / (float)groups;
    pdl_leave();
}

struct BackArgs {
    const int32_t *ids, *counts;
    const float *lse, *live, *dweights, *dloss;
    void *dlogits;
    uint64_t stride;
    bool vec;
};

// Tokens of a warp's ring in the backward pass (three to six take the same time), and the bytes of one: the row, its
// ids, the gradients of its weights, its log-sum-exp.
constexpr int kRing = 4;
template <class T, int PER>
__host__ __device__ constexpr uint32_t ring_slot() {
    return 32 * PER * (uint32_t)sizeof(T) + 128 + 128 + 16;
}
// bf16 and a vector a lane: 262144 x 256 98 us through registers, 76 us through the ring. FP32 with a vector a lane: 68
// against 72 us; two vectors: the ring is more than a launch gives without asking.
template <class T, int PER>
__host__ __device__ constexpr bool has_ring() {
    return PER == 8 && sizeof(T) == 2;
}
__device__ __forceinline__ void copy_async4(void *smem, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src) : "memory");
}

// Saved log-sum-exps below this are taken as they are: their rounding is at most 2^-21, the exponents' own. Beside a
// maximum far from 0 an FP32 number has no room for the sum's logarithm; there the probabilities are divided by
// their sum (262144 x 256 bf16 75 us either way, 85 us where all tokens are far).
constexpr float kFar = 16.f;

// What the choices add to their experts' elements goes through a row of shared
// memory of the warp's own, all zeros between two tokens.
// RING: a lane's run is one 16-byte vector; tokens come through a ring of the warp's own, copied kRing
// tokens ahead, and a choice's logit is looked up there. Else they come through registers, two ahead.
template <class T, int PER, bool RING>
__global__ void __launch_bounds__(kThreads, back_resident(PER)) k_balance_backward(const Args a, const BackArgs q) {
    extern __shared__ __align__(128) float sm_extra[];   // [warps][32 PER], then RING: [warps][kRing] slots
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *extras = sm_extra + warp * 32 * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) extras[lane + 32 * i] = 0.f;
    __syncwarp();
    pdl_enter();
    const uint64_t warps = (uint64_t)gridDim.x * kWarps, me = (uint64_t)blockIdx.x * kWarps + warp;
    // each warp a run of tokens, so that its group seldom changes
    const uint64_t t0 = a.tokens / warps * me + a.tokens % warps * me / warps;
    const uint64_t t1 = a.tokens / warps * (me + 1) + a.tokens % warps * (me + 1) / warps;
    const float dloss = q.dloss ? *q.dloss : 1.f;
    const T *logits = reinterpret_cast<const T *>(a.logits);
    const bool chooses = lane < a.k && q.dweights;
    uint64_t group = t0 < t1 ? t0 / a.per_group : 0, left = 0;   // left: tokens before the next group
    if (t0 < t1) left = (group + 1) * a.per_group - t0;
    bool fresh = true;
    float f[PER], ab = 0.f, two_z = 0.f;
    // A token's numbers are asked for two tokens ahead, its ids three, its chosen logits two.
    float lse_next = 0.f, up_next = 0.f, zid_next = 0.f, lse_2 = 0.f, up_2 = 0.f, zid_2 = 0.f;
    RunOf<T, PER> ahead, run_2;
    int32_t id_next = -1, id_2 = -1, id_3 = -1;
    const T *row = logits + t0 * a.stride;
    const float *lse_from = q.lse + t0, *up_from = chooses ? q.dweights + t0 * a.k + lane : nullptr;
    const int32_t *id_from = chooses ? q.ids + t0 * a.k + lane : nullptr;
    T *out = reinterpret_cast<T *>(q.dlogits) + t0 * q.stride;
    const uint32_t tokens = (uint32_t)(t1 - t0);
    uint32_t ids_left = tokens, to_fetch = tokens;
    auto next_id = [&]() {
        if (ids_left == 0 || !chooses) return -1;
        --ids_left;
        const int32_t id = *id_from;   // looked at when it has had time to come
        id_from += a.k;
        return id;
    };
    auto fetch = [&]() {
        lse_next = lse_2, up_next = up_2, zid_next = zid_2, ahead = run_2, id_next = id_2;
        id_2 = id_3, id_3 = next_id();
        if (to_fetch == 0) return;
        --to_fetch;
        lse_2 = *lse_from++;
        run_2 = load_run<T, PER>(row, a.experts, lane, a.vec);
        zid_2 = up_2 = 0.f;
        if ((uint32_t)id_2 >= a.experts) id_2 = -1;
        if (id_2 >= 0) zid_2 = to_f32(row[id_2]), up_2 = *up_from;
        row += a.stride;
        if (chooses) up_from += a.k;
    };
    char *ring = reinterpret_cast<char *>(sm_extra + kThreads * PER) + warp * kRing * ring_slot<T, PER>();
    uint32_t slot = 0, copy_slot = 0;
    constexpr uint32_t kRow = 32 * PER * sizeof(T), kRun = PER * sizeof(T);
    auto fill = [&]() {
        if (to_fetch != 0) {
            --to_fetch;
            char *to = ring + copy_slot * ring_slot<T, PER>();
            if (lane * PER < a.experts) {
#pragma unroll
                for (uint32_t i = 0; i < kRun; i += 16) copy_async16(to + lane * kRun + i, reinterpret_cast<const char *>(row + lane * PER) + i);
            }
            if (chooses) copy_async4(to + kRow + lane * 4, id_from), copy_async4(to + kRow + 128 + lane * 4, up_from);
            if (lane == 0) copy_async4(to + kRow + 256, lse_from);
            row += a.stride, ++lse_from;
            if (chooses) id_from += a.k, up_from += a.k;
        }
        copy_commit();
        copy_slot = copy_slot + 1 == kRing ? 0 : copy_slot + 1;
    };
    if constexpr (RING) {
        for (int i = 0; i < kRing; ++i) fill();
    } else {
        id_3 = next_id();
        fetch();
        fetch();
    }
    for (uint32_t todo = tokens; todo != 0; --todo, out += q.stride) {
        float z[PER], lse, up = 0.f, zid = 0.f;
        int32_t id = -1;
        if constexpr (RING) {
            copy_wait<kRing - 1>();
            __syncwarp();
            const char *from = ring + slot * ring_slot<T, PER>();
            lse = *reinterpret_cast<const float *>(from + kRow + 256);
            if (chooses) {
                id = *reinterpret_cast<const int32_t *>(from + kRow + lane * 4);
                up = *reinterpret_cast<const float *>(from + kRow + 128 + lane * 4);
                if ((uint32_t)id >= a.experts) id = -1;
                if (id >= 0) zid = to_f32(reinterpret_cast<const T *>(from)[id]);
            }
            RunOf<T, PER> run;
#pragma unroll
            for (uint32_t i = 0; i < kRun / 4; i += 4) {
                constexpr uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;   // -inf
                const uint4 v = lane * PER < a.experts ? *reinterpret_cast<const uint4 *>(from + lane * kRun + i * 4)
                                                       : make_uint4(none, none, none, none);
                run.w[i] = v.x, run.w[i + 1] = v.y, run.w[i + 2] = v.z, run.w[i + 3] = v.w;
            }
            unpack_run<T, PER>(run, z);
            __syncwarp();
            fill();
            slot = slot + 1 == kRing ? 0 : slot + 1;
        } else {
            lse = lse_next, up = up_next, zid = zid_next, id = id_next;
            unpack_run<T, PER>(ahead, z);
            fetch();
        }
        if (fresh) {
            fresh = false;
            const float n = q.live[group], scale = dloss / ((float)a.groups * n), share = (float)a.experts / ((float)a.k * n);
            ab = a.balance_weight * scale, two_z = 2.f * a.z_weight * scale;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t e = lane * PER + i;
                f[i] = e < a.experts ? ab * share * (float)q.counts[group * a.experts + e] : 0.f;
            }
        }
        if (--left == 0) ++group, left = a.per_group, fresh = true;
        if (lse == -INFINITY) {   // masked
#pragma unroll
            for (int i = 0; i < PER; ++i) z[i] = 0.f;
            store_run<T, PER>(out, a.experts, lane, q.vec, z);
            continue;
        }
        float s;
        if constexpr (PER == 1) {
            z[0] = ex2((z[0] - lse) * kLog2e);
            s = f[0] * z[0];
        } else {
            float2 s2 = both(0.f);
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 d = mul2(add2(make_float2(z[i], z[i + 1]), both(-lse)), both(kLog2e));
                z[i] = ex2(d.x), z[i + 1] = ex2(d.y);
                s2 = fma2(make_float2(f[i], f[i + 1]), make_float2(z[i], z[i + 1]), s2);
            }
            s = s2.x + s2.y;
        }
        float scale = 1.f;
        if (!(fabsf(lse) < kFar)) {   // the same in all lanes
            float total = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) total += z[i];
            scale = reciprocal(warp_sum(total));
#pragma unroll
            for (int i = 0; i < PER; ++i) z[i] *= scale;
            s *= scale;
        }
        float extra = 0.f, dot = 0.f;
        if (q.dweights) {
            const float p = id >= 0 ? ex2((zid - lse) * kLog2e) * scale : 0.f, pu = p * up;
            dot = warp_sum(pu);
            if (a.renormalise) {
                // w (u - sum w u), w = p / sum: as p / sum^2 (u sum - sum p u), whose difference is 0 to the bit where one
                // choice has all the weight (two roundings of one product: no fused multiply-add)
                const float sum = warp_sum(p), inv = reciprocal(sum);
                extra = p * inv * (inv * __fsub_rn(__fmul_rn(up, sum), dot)), dot = 0.f;
            } else {
                extra = pu;
            }
            if (id >= 0) extras[id] = extra;
        }
        const float rest = two_z * lse - warp_sum(s) - dot;
        // p (f + rest), and what the choices add
        if (q.dweights) __syncwarp();
        if constexpr (PER == 1) {
            z[0] = fmaf(z[0], f[0] + rest, q.dweights ? extras[lane] : 0.f);
        } else {
            const float2 *more = reinterpret_cast<const float2 *>(extras + lane * PER);
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 r = fma2(make_float2(z[i], z[i + 1]), add2(make_float2(f[i], f[i + 1]), both(rest)),
                                      q.dweights ? more[i / 2] : both(0.f));
                z[i] = r.x, z[i + 1] = r.y;
            }
        }
        if (q.dweights) {
            __syncwarp();
            if (id >= 0) extras[id] = 0.f;
            __syncwarp();
        }
        store_run<T, PER>(out, a.experts, lane, q.vec, z);
    }
    pdl_leave();
}

// ---------------------------------------------------------------------- host

int bad(const char *m) { return fail(BF16OPT_ERR_INVALID_ARG, std::string("balance: ") + m); }

int check(const bf16opt_balance_t *d) {
    if (!d) return bad("the descriptor is NULL");
    if (!type_ok(d->logits_type)) return bad("unknown element type");
    if (d->experts < 1 || d->experts > BF16OPT_BALANCE_MAX_EXPERTS) return bad("experts must lie in [1, BF16OPT_BALANCE_MAX_EXPERTS]");
    if (d->k < 1 || d->k > d->experts || d->k > BF16OPT_BALANCE_MAX_K) return bad("k must lie in [1, min(experts, BF16OPT_BALANCE_MAX_K)]");
    if (d->groups < 1 || d->tokens % d->groups != 0 || (d->tokens && d->groups > d->tokens)) return bad("groups must divide tokens");
    if (d->tokens >= (1ull << 40) || d->groups >= (1ull << 40)) return bad("too many tokens");
    if (d->tokens / d->groups >= (1ull << 31)) return bad("a group has 2^31 tokens or more");
    if (d->logits_stride < d->experts) return bad("a row stride is below experts");
    if (d->renormalise != 0 && d->renormalise != 1) return bad("renormalise must be 0 or 1");
    if (!(std::isfinite(d->balance_weight) && d->balance_weight >= 0.f) || !(std::isfinite(d->z_weight) && d->z_weight >= 0.f))
        return bad("balance_weight and z_weight must be finite and >= 0");
    uint64_t n = 0;
    if (!span_bytes(d->tokens, d->logits_stride, d->experts, type_bytes(d->logits_type), n)) return bad("the sizes overflow");
    return BF16OPT_OK;
}

// CTAs of the forward pass: four per SM, each with at least 64 tokens.
uint32_t teams_of(const bf16opt_balance_t *d, int sms) {
    return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>((uint64_t)sms * 4, d->tokens / 64));
}
uint64_t workspace_floats(const bf16opt_balance_t *d, uint32_t teams) {
    return teams == 1 ? 0 : (d->groups + 3) / 4 * 4 + 2 * (uint64_t)teams * slot_floats(d->experts);
}

int per_of(uint32_t experts) {
    int p = 1;
    while (p * 32 < (int)experts) p *= 2;
    return p;
}

Args args_of(const bf16opt_balance_t *d) {
    Args a = {};
    a.tokens = d->tokens, a.groups = d->groups, a.per_group = d->tokens / d->groups;
    a.experts = d->experts, a.k = d->k, a.renormalise = d->renormalise;
    a.logits = d->logits, a.stride = d->logits_stride;
    a.mask = d->mask, a.balance_weight = d->balance_weight, a.z_weight = d->z_weight;
    return a;
}

// Whether a lane's run of `per` elements is one aligned run in every row.
bool runs(const void *p, uint64_t stride, uint32_t experts, int per, uint64_t elem) {
    const uint64_t run = std::min<uint64_t>(16, per * elem);
    return experts % per == 0 && !misaligned(p, run) && stride * elem % run == 0;
}

template <class F>
int by_per(int per, F &&f) {
    switch (per) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
    }
}

int done(cudaError_t e) { return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "balance kernel launch"); }

int workspace(const bf16opt_balance_t *d, uint64_t *bytes) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    const int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    if (!bytes) return bad("bytes is NULL");
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "balance: no CUDA device");
    *bytes = workspace_floats(d, teams_of(d, sms)) * 4;
    return BF16OPT_OK;
}

struct Part {
    const void *p;
    uint64_t n;
};
bool apart(std::initializer_list<Part> outs, std::initializer_list<Part> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Part &x : ins)
            if (overlap(o->p, o->n, x.p, x.n)) return false;
        for (auto e = outs.begin(); e != o; ++e)
            if (overlap(o->p, o->n, e->p, e->n)) return false;
    }
    return true;
}

int forward(const bf16opt_balance_t *d, int32_t *ids, float *weights, int32_t *counts, float *loss, float *saved, void *ws,
            uint64_t ws_bytes, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    const int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    if (!counts || !loss || !saved || (d->tokens && (!d->logits || !ids || !weights))) return bad("a pointer is NULL");
    const uint64_t elem = type_bytes(d->logits_type);
    if (misaligned(d->logits, elem) || misaligned(ids, 4) || misaligned(weights, 4) || misaligned(counts, 4) ||
        misaligned(loss, 4) || misaligned(saved, 4) || misaligned(ws, 16))
        return fail(BF16OPT_ERR_ALIGNMENT, "balance: a pointer is not aligned to its element (workspace: 16 bytes)");
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "balance: no CUDA device");
    const cudaStream_t st = (cudaStream_t)stream;
    const uint64_t cb = d->groups * d->experts * 4, tk = d->tokens * d->k * 4;
    if (d->tokens == 0) {
        cudaError_t e = cudaMemsetAsync(counts, 0, cb, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(loss, 0, 4, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(saved, 0, d->groups * 4, st);
        return done(e);
    }
    const uint32_t teams = teams_of(d, sms);
    const uint64_t need = workspace_floats(d, teams) * 4;
    if (need && (!ws || ws_bytes < need)) return bad("the workspace is too small");
    uint64_t zb = 0;
    span_bytes(d->tokens, d->logits_stride, d->experts, elem, zb);
    if (!apart({{ids, tk}, {weights, tk}, {counts, cb}, {loss, 4}, {saved, (d->tokens + d->groups) * 4}, {ws, need}},
               {{d->logits, zb}, {d->mask, d->tokens}}))
        return bad("an output overlaps an input or another output");
    Args a = args_of(d);
    a.ids = ids, a.weights = weights, a.counts = counts, a.loss = loss, a.lse = saved, a.live = saved + d->tokens;
    a.group_loss = (float *)ws, a.slots = (float *)ws + (d->groups + 3) / 4 * 4, a.teams = teams;
    const int per = per_of(d->experts);
    a.vec = runs(d->logits, d->logits_stride, d->experts, per, elem);
    const size_t smem = (kWarps + 1) * (size_t)d->experts * 4;
    int r = by_per(per, [&](auto p) {
        constexpr int PER = decltype(p)::value;
        Launch l{teams, (unsigned)kThreads, smem, st, 0, true};
        return done(d->logits_type == BF16OPT_TYPE_BF16 ? launch(l, k_balance_forward<__nv_bfloat16, PER>, a)
                                                        : launch(l, k_balance_forward<float, PER>, a));
    });
    if (r != BF16OPT_OK || teams == 1) return r;
    if (d->groups <= 64) {   // few groups: one cluster joins them and adds up their losses
        const unsigned cluster = (uint64_t)teams * d->experts >= 8192 || d->groups > 1 ? 8 : 1;
        Launch l{cluster, 32 * kJoinWarps, 0, st, cluster, true};
        return done(launch(l, k_balance_join<true>, a));
    }
    Launch l{(unsigned)std::min<uint64_t>(d->groups, 1024), 32 * kJoinWarps, 0, st, 0, true};
    r = done(launch(l, k_balance_join<false>, a));
    if (r != BF16OPT_OK) return r;
    Launch l2{1, (unsigned)kThreads, 0, st, 0, true};
    return done(launch(l2, k_balance_sum, (const float *)a.group_loss, a.groups, loss));
}

int backward(const bf16opt_balance_t *d, const int32_t *ids, const int32_t *counts, const float *saved, const float *dweights,
             const float *dloss, void *dlogits, uint64_t dlogits_stride, void *stream) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    const int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    if (dlogits_stride < d->experts) return bad("a row stride is below experts");
    if (d->tokens == 0) return BF16OPT_OK;
    if (!d->logits || !ids || !counts || !saved || !dlogits) return bad("a pointer is NULL");
    const uint64_t elem = type_bytes(d->logits_type);
    if (misaligned(d->logits, elem) || misaligned(dlogits, elem) || misaligned(ids, 4) || misaligned(counts, 4) ||
        misaligned(saved, 4) || misaligned(dweights, 4) || misaligned(dloss, 4))
        return fail(BF16OPT_ERR_ALIGNMENT, "balance: a pointer is not aligned to its element");
    uint64_t zb = 0, gb = 0;
    span_bytes(d->tokens, d->logits_stride, d->experts, elem, zb);
    if (!span_bytes(d->tokens, dlogits_stride, d->experts, elem, gb)) return bad("the sizes overflow");
    const uint64_t tk = d->tokens * d->k * 4;
    const bool in_place = dlogits == d->logits && dlogits_stride == d->logits_stride;
    if (!apart({{dlogits, gb}}, {{in_place ? nullptr : d->logits, zb}, {ids, tk}, {counts, d->groups * d->experts * 4},
                                 {saved, (d->tokens + d->groups) * 4}, {dweights, tk}, {dloss, 4}}))
        return bad("an output overlaps an input");
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "balance: no CUDA device");
    Args a = args_of(d);
    BackArgs q;
    q.ids = ids, q.counts = counts, q.lse = saved, q.live = saved + d->tokens, q.dweights = dweights, q.dloss = dloss;
    q.dlogits = dlogits, q.stride = dlogits_stride;
    const int per = per_of(d->experts);
    a.vec = runs(d->logits, d->logits_stride, d->experts, per, elem);
    q.vec = runs(dlogits, dlogits_stride, d->experts, per, elem);
    const unsigned grid = (unsigned)std::min<uint64_t>((d->tokens + kWarps - 1) / kWarps, (uint64_t)sms * back_resident(per));
    return by_per(per, [&](auto p) {
        constexpr int PER = decltype(p)::value;
        auto go = [&](auto *type) {
            using T = std::remove_pointer_t<decltype(type)>;
            Launch l{grid, (unsigned)kThreads, (size_t)kThreads * PER * 4, (cudaStream_t)stream, 0, true};
            if constexpr (has_ring<T, PER>())
                if (a.vec) {
                    l.smem += (size_t)kWarps * kRing * ring_slot<T, PER>();
                    return done(launch(l, k_balance_backward<T, PER, true>, a, q));
                }
            return done(launch(l, k_balance_backward<T, PER, false>, a, q));
        };
        return d->logits_type == BF16OPT_TYPE_BF16 ? go((__nv_bfloat16 *)nullptr) : go((float *)nullptr);
    });
}

}  // namespace
}  // namespace bf16ops

extern "C" int bf16opt_balance_workspace(const bf16opt_balance_t *d, uint64_t *bytes) {
    return bf16ops::guarded([&] { return bf16ops::workspace(d, bytes); });
}

extern "C" int bf16opt_balance_forward(const bf16opt_balance_t *d, int32_t *ids, float *weights, int32_t *counts, float *loss,
                                       float *saved, void *workspace, uint64_t workspace_bytes, void *stream) {
    return bf16ops::guarded(
        [&] { return bf16ops::forward(d, ids, weights, counts, loss, saved, workspace, workspace_bytes, stream); });
}

extern "C" int bf16opt_balance_backward(const bf16opt_balance_t *d, const int32_t *ids, const int32_t *counts,
                                        const float *saved, const float *dweights, const float *dloss, void *dlogits,
                                        uint64_t dlogits_stride, void *stream) {
    return bf16ops::guarded(
        [&] { return bf16ops::backward(d, ids, counts, saved, dweights, dloss, dlogits, dlogits_stride, stream); });
}
