// norm_gate.cu -- the norms before and after a block with its gate and residual
// scale, forward and backward (bf16opt_norm_gate_* of include/bf16opt.h).
//
// Forward: one CTA (or one warp, for short rows) holds a row of x and y in
// registers, so both are read once and r and h written once.
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
#include <cooperative_groups.h>

#include <algorithm>

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

// Weights: read again and again, so kept in L1.
template <bool VEC>
__device__ __forceinline__ void load8_weight(const void *w, int type, uint32_t n, uint32_t slot, uint32_t threads, uint32_t t,
                                             float none, float (&f)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = none;
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

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + ex2(-x * kLog2e)); }

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
k_norm_forward(const Args a, const TS *x, const TB *y, TS *r, TB *h, float *stats) {
    __shared__ float buf[64];
    const uint32_t threads = WARP ? 32u : blockDim.x, t = WARP ? threadIdx.x & 31u : threadIdx.x;
    const uint32_t n = a.hidden;
    uint32_t turn = 0;
    pdl_enter();
    const uint64_t row = WARP ? (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
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

// ----------------------------------------------------------------------- backward

constexpr int kColumns = 4096;   // columns of one CTA: 512 threads of 8
constexpr int kSums = 8;

struct BackArgs {
    const void *dr, *dh, *r, *y;
    const float *stats;
    void *dx, *dy, *dgate;
    // FP32 partial sums: [teams][4][hidden] of the weights' gradients, and
    // [2 teams][hidden] of the gates' that straddle teams
    float *part, *gate_part;
    uint32_t teams;
    bool need_weights, shared_gate;   // shared_gate: rows share gate rows and dgate is wanted
};

// Rows [first(p), first(p + 1)) are team p's.
__host__ __device__ inline uint64_t team_row(uint64_t rows, uint32_t teams, uint32_t p) {
    return rows / teams * p + rows % teams * p / teams;
}

// The team of a row.
__device__ __forceinline__ uint32_t team_of(uint64_t rows, uint32_t teams, uint64_t row) {
    uint32_t p = (uint32_t)(row / (rows / teams + 1));   // not beyond it
    while (team_row(rows, teams, p + 1) <= row) ++p;
    return p;
}

// Sum of eight values over a warp: each step a lane keeps half of the values
// and hands the other half over, so it costs 9 shuffles, not 40.  Lane l ends up
// with the sum of value (l & 7) reversed in bits -- see lane_value.
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

template <class TB, class TS, bool VEC>
__global__ void __launch_bounds__(512, 1) k_norm_backward(const Args a, const BackArgs q) {
    // [2][CTAs of the cluster][8 sums]
    __shared__ float sm_sums[2][16][kSums];        // [turn][warp]
    __shared__ float sm_cluster[2][4][kSums];      // [turn][rank]
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t threads = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = threads / 32;
    const uint32_t team = blockIdx.x / ranks;
    // this CTA's columns: [c0, c0 + n)
    const uint32_t c0 = rank * threads * 8;
    const uint32_t n = c0 < a.hidden ? min(a.hidden - c0, threads * 8) : 0u;
    const float inv_h = 1.f / (float)a.hidden;
    const bool pre = a.pre.kind != BF16OPT_NORM_NONE, post = a.post.kind != BF16OPT_NORM_NONE;
    const bool pre_layer = a.pre.kind == BF16OPT_NORM_LAYER, post_layer = a.post.kind == BF16OPT_NORM_LAYER;
    pdl_enter();
    if (ranks > 1) cluster.sync();

    const uint32_t wb = a.weight_type == BF16OPT_TYPE_BF16 ? 2 : 4;
    auto at = [&](const void *w) { return w ? (const void *)((const char *)w + (size_t)c0 * wb) : nullptr; };
    const void *w1p = at(a.pre.weight), *w2p = at(a.post.weight), *b2p = at(a.post.bias);

    float dw1[8] = {}, db1[8] = {}, dw2[8] = {}, db2[8] = {}, dg[8] = {};
    const uint64_t row0 = team_row(a.rows, q.teams, team), row1 = team_row(a.rows, q.teams, team + 1);
    uint64_t group = a.gate ? row0 / a.rows_per_gate : 0;
    uint32_t turn = 0;
    for (uint64_t row = row0; row < row1; ++row, ++turn) {
        const uint64_t o = row * a.hidden + c0;
        float r8[8], y8[8], dr8[8], dh8[8], g8[8], w1[8], w2[8];
        const float mu1 = pre ? q.stats[4 * row] : 0.f, rs1 = pre ? q.stats[4 * row + 1] : 0.f;
        const float mu2 = post ? q.stats[4 * row + 2] : 0.f, rs2 = post ? q.stats[4 * row + 3] : 1.f;
        load8<VEC>(reinterpret_cast<const TB *>(q.y) + o, n, 0, threads, t, y8);
        if (q.dr) load8<VEC>(reinterpret_cast<const TS *>(q.dr) + o, n, 0, threads, t, dr8);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) dr8[i] = 0.f;
        if (pre && q.dh) {
            load8<VEC>(reinterpret_cast<const TS *>(q.r) + o, n, 0, threads, t, r8);
            load8<VEC>(reinterpret_cast<const TB *>(q.dh) + o, n, 0, threads, t, dh8);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r8[i] = mu1, dh8[i] = 0.f;
        }
        if (a.gate) load8<VEC>(reinterpret_cast<const TB *>(a.gate) + row / a.rows_per_gate * a.hidden + c0, n, 0, threads, t, g8);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) g8[i] = 1.f;
        load8_weight<VEC>(w1p, a.weight_type, n, 0, threads, t, 1.f, w1);
        load8_weight<VEC>(w2p, a.weight_type, n, 0, threads, t, 1.f, w2);

        float s[kSums] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = column<VEC>(0, threads, t, i) < n;
            const float xhat = in ? (r8[i] - mu1) * rs1 : 0.f, yhat = in ? (y8[i] - mu2) * rs2 : 0.f;
            const float av = w1[i] * dh8[i];
            const float base = fmaf(rs1, av, dr8[i]);
            float act = g8[i];
            if (a.gate_act == BF16OPT_GATE_SIGMOID && a.gate) act = sigmoid(act);
            const float c = in ? a.branch_scale * w2[i] * act : 0.f;
            s[0] += av;
            s[1] = fmaf(av, xhat, s[1]);
            s[2] = fmaf(c, base, s[2]);
            s[3] += c;
            s[4] = fmaf(c, xhat, s[4]);
            const float cy = c * yhat;
            s[5] = fmaf(cy, base, s[5]);
            s[6] += cy;
            s[7] = fmaf(cy, xhat, s[7]);
        }
        const float mine = warp_sum8(s, lane);
        if (lane < 8) sm_sums[turn & 1][warp][lane_value(lane)] = mine;
        __syncthreads();
        if (ranks > 1) {
            if (t < ranks * kSums) {
                float v = 0.f;
                for (uint32_t i = 0; i < warps; ++i) v += sm_sums[turn & 1][i][t & 7];
                *cluster.map_shared_rank(&sm_cluster[turn & 1][rank][t & 7], t >> 3) = v;
            }
            cluster.sync();
        }
#pragma unroll
        for (int k = 0; k < kSums; ++k) s[k] = 0.f;
        if (ranks > 1) {
            for (uint32_t i = 0; i < ranks; ++i)
#pragma unroll
                for (int k = 0; k < kSums; ++k) s[k] += sm_cluster[turn & 1][i][k];
        } else {
            for (uint32_t i = 0; i < warps; ++i)
#pragma unroll
                for (int k = 0; k < kSums; ++k) s[k] += sm_sums[turn & 1][i][k];
        }
        // g = base - rs1 (m1 + xhat m2);  e = c g;  dy = rs2 (e - n1 - yhat n2)
        const float m1 = pre_layer ? s[0] * inv_h * rs1 : 0.f, m2 = s[1] * inv_h * rs1;
        const float n1 = post_layer ? (s[2] - m1 * s[3] - m2 * s[4]) * inv_h : 0.f;
        const float n2 = post ? (s[5] - m1 * s[6] - m2 * s[7]) * inv_h : 0.f;

        if (a.gate && q.shared_gate && row / a.rows_per_gate != group) {   // the gate's rows end: its sum is whole if they began here
            const bool began = group * a.rows_per_gate >= row0;
            if (began) store8<VEC>(reinterpret_cast<TB *>(q.dgate) + group * a.hidden + c0, n, 0, threads, t, dg);
            else store8<VEC>(q.gate_part + (size_t)(2 * team) * a.hidden + c0, n, 0, threads, t, dg);
#pragma unroll
            for (int i = 0; i < 8; ++i) dg[i] = 0.f;
            group = row / a.rows_per_gate;
        }
        float b2[8];
        load8_weight<VEC>(b2p, a.weight_type, n, 0, threads, t, 0.f, b2);
        float dx8[8], dy8[8], dgr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = column<VEC>(0, threads, t, i) < n;
            const float xhat = in ? (r8[i] - mu1) * rs1 : 0.f, yhat = in ? (y8[i] - mu2) * rs2 : 0.f;
            const float base = fmaf(rs1, w1[i] * dh8[i], dr8[i]);
            const float g = base - fmaf(xhat, m2, m1);
            dx8[i] = a.residual_scale * g;
            const float du = a.branch_scale * g;
            float act = g8[i], slope = 1.f;
            if (a.gate_act == BF16OPT_GATE_SIGMOID && a.gate) {
                act = sigmoid(act);
                slope = act * (1.f - act);
            }
            dgr[i] = slope * du * fmaf(yhat, w2[i], b2[i]);
            const float dn = act * du;
            dw2[i] = fmaf(dn, yhat, dw2[i]);
            db2[i] += dn;
            dw1[i] = fmaf(dh8[i], xhat, dw1[i]);
            db1[i] += dh8[i];
            dy8[i] = post ? rs2 * (fmaf(w2[i], dn, -n1) - yhat * n2) : dn;
        }
        store8<VEC>(reinterpret_cast<TS *>(q.dx) + o, n, 0, threads, t, dx8);
        store8<VEC>(reinterpret_cast<TB *>(q.dy) + o, n, 0, threads, t, dy8);
        if (a.gate && q.dgate) {
            if (q.shared_gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i) dg[i] += dgr[i];
            } else {
                store8<VEC>(reinterpret_cast<TB *>(q.dgate) + o, n, 0, threads, t, dgr);
            }
        }
    }
    if (q.shared_gate && row0 < row1) {
        const bool began = group * a.rows_per_gate >= row0, ends = (group + 1) * a.rows_per_gate <= row1;
        if (began && ends) store8<VEC>(reinterpret_cast<TB *>(q.dgate) + group * a.hidden + c0, n, 0, threads, t, dg);
        else store8<VEC>(q.gate_part + (size_t)(2 * team + (began && group != row0 / a.rows_per_gate)) * a.hidden + c0, n, 0, threads, t, dg);
    }
    if (q.need_weights) {
        float *p = q.part + (size_t)team * 4 * a.hidden + c0;
        store8<VEC>(p, n, 0, threads, t, dw1);
        store8<VEC>(p + a.hidden, n, 0, threads, t, db1);
        store8<VEC>(p + 2 * (size_t)a.hidden, n, 0, threads, t, dw2);
        store8<VEC>(p + 3 * (size_t)a.hidden, n, 0, threads, t, db2);
    }
}

// The partial sums joined, in the teams' order: 32 columns by 8 runs of teams.
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
__global__ void __launch_bounds__(256) k_norm_join(const JoinArgs j) {
    __shared__ float sm[8][32];
    pdl_enter();
    const uint32_t lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const uint32_t c = blockIdx.x * 32 + lane;
    for (uint64_t b = blockIdx.y; b < 4 + (j.dgate ? j.gate_rows : 0); b += gridDim.y) {
        const float *p;          // part i is p + i * stride (+ skip for i = 0)
        size_t stride, skip = 0;
        uint32_t count;
        uint64_t at = c;
        void *out;
        if (b < 4) {
            out = j.out[b];
            p = j.part + b * j.hidden, stride = 4 * (size_t)j.hidden, count = j.teams;
        } else {
            const uint64_t g = b - 4, first = g * j.rows_per_gate, last = first + j.rows_per_gate - 1;
            uint32_t p0 = team_of(j.rows, j.teams, first), p1 = team_of(j.rows, j.teams, last);
            out = p0 == p1 ? nullptr : j.dgate;   // within one team: already written
            at = g * j.hidden + c;
            p = j.gate_part + (size_t)(2 * p0) * j.hidden, stride = 2 * (size_t)j.hidden, count = p1 - p0 + 1;
            skip = first > team_row(j.rows, j.teams, p0) ? j.hidden : 0;   // the first team's last gate, not its first
        }
        if (!out) continue;
        float s = 0.f;
        const uint32_t i0 = (uint32_t)((uint64_t)count * run / 8), i1 = (uint32_t)((uint64_t)count * (run + 1) / 8);
        if (c < j.hidden)
            for (uint32_t i = i0; i < i1; ++i) s += p[i * stride + (i ? 0 : skip) + c];
        sm[run][lane] = s;
        __syncthreads();
        if (run == 0 && c < j.hidden) {
            for (int i = 1; i < 8; ++i) s += sm[i][lane];
            store_typed(out, b < 4 ? j.weight_type : j.gate_type, at, s);
        }
        __syncthreads();
    }
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

template <class TB, class TS, bool VEC>
int forward_v(const Args &a, const void *x, const void *y, void *r, void *h, float *stats, cudaStream_t st) {
    const uint32_t vecs = (a.hidden + 7) / 8;
    auto go = [&](auto kernel, unsigned block, bool warp) {
        Launch l{(unsigned)(warp ? (a.rows + 3) / 4 : a.rows), block, 0, st, 0, true};
        const cudaError_t e = launch(l, kernel, a, (const TS *)x, (const TB *)y, (TS *)r, (TB *)h, stats);
        return e == cudaSuccess ? BF16OPT_OK : fail_cuda(e, "norm_gate kernel launch");
    };
    if (vecs <= 32) return go(k_norm_forward<TB, TS, VEC, true, 1>, 128, true);
    if (vecs <= 64) return go(k_norm_forward<TB, TS, VEC, true, 2>, 128, true);
    auto block = [&](uint32_t nv) { return (unsigned)(((vecs + nv - 1) / nv + 31) / 32 * 32); };
    if (vecs <= 512) return go(k_norm_forward<TB, TS, VEC, false, 1>, block(1), false);
    if (vecs <= 1024) return go(k_norm_forward<TB, TS, VEC, false, 2>, block(2), false);
    return go(k_norm_forward<TB, TS, VEC, false, 4>, block(4), false);
}

// The backward pass's shape, from the sizes and the device alone.
struct Shape {
    unsigned cluster, threads;
    uint32_t teams;
    uint64_t part_floats, gate_floats;
};
Shape shape_of(const bf16opt_norm_gate_t *d, int sms) {
    Shape s;
    s.cluster = (d->hidden + kColumns - 1) / kColumns;
    if (s.cluster == 3) s.cluster = 4;
    const uint32_t cols = (d->hidden + s.cluster - 1) / s.cluster;
    s.threads = ((cols + 7) / 8 + 31) / 32 * 32;
    const uint64_t teams = std::max<uint64_t>(1, (uint64_t)sms * std::max(1u, 512 / s.threads) / s.cluster);
    s.teams = (uint32_t)std::min<uint64_t>(teams, std::max<uint64_t>(1, d->rows));
    s.part_floats = (uint64_t)s.teams * 4 * d->hidden;
    s.gate_floats = d->gate_rows && d->gate_rows != d->rows ? (uint64_t)s.teams * 2 * d->hidden : 0;
    return s;
}

template <class TB, class TS, bool VEC>
int backward_v(const Args &a, const BackArgs &q, const Shape &s, cudaStream_t st) {
    Launch l{s.teams * s.cluster, s.threads, 0, st, s.cluster, true};
    const cudaError_t e = launch(l, k_norm_backward<TB, TS, VEC>, a, q);
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
    using B = __nv_bfloat16;
    if (d->branch_type == BF16OPT_TYPE_F32)
        return vec ? forward_v<float, float, true>(a, x, y, r, h, stats, st) : forward_v<float, float, false>(a, x, y, r, h, stats, st);
    if (d->stream_type == BF16OPT_TYPE_F32)
        return vec ? forward_v<B, float, true>(a, x, y, r, h, stats, st) : forward_v<B, float, false>(a, x, y, r, h, stats, st);
    return vec ? forward_v<B, B, true>(a, x, y, r, h, stats, st) : forward_v<B, B, false>(a, x, y, r, h, stats, st);
}

int workspace(const bf16opt_norm_gate_t *d, uint64_t *bytes) {
    bf16opt_fail_unbound(BF16OPT_OK, "");
    const int rc = check(d);
    if (rc != BF16OPT_OK) return rc;
    if (!bytes) return fail(BF16OPT_ERR_INVALID_ARG, "norm_gate: bytes is NULL");
    const int sms = sm_count();
    if (sms < 1) return fail(BF16OPT_ERR_UNSUPPORTED, "norm_gate: no CUDA device");
    const Shape s = shape_of(d, sms);
    *bytes = (s.part_floats + s.gate_floats) * 4;
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
    bool need = false;
    for (void *w : outs) {
        need = need || w;
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
    const Shape s = shape_of(d, sms);
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
    q.teams = s.teams, q.need_weights = need;
    q.shared_gate = dgate && d->gate_rows != d->rows;
    const bool vec = vectors(d, {dr, dh, r, y, dx, dy, dgate});
    using B = __nv_bfloat16;
    if (d->branch_type == BF16OPT_TYPE_F32)
        rc = vec ? backward_v<float, float, true>(a, q, s, st) : backward_v<float, float, false>(a, q, s, st);
    else if (d->stream_type == BF16OPT_TYPE_F32)
        rc = vec ? backward_v<B, float, true>(a, q, s, st) : backward_v<B, float, false>(a, q, s, st);
    else
        rc = vec ? backward_v<B, B, true>(a, q, s, st) : backward_v<B, B, false>(a, q, s, st);
    if (rc != BF16OPT_OK || (!need && !q.shared_gate)) return rc;
    JoinArgs j;
    j.part = q.part, j.gate_part = q.gate_part;
    for (int i = 0; i < 4; ++i) j.out[i] = outs[i];
    j.weight_type = d->weight_type, j.gate_type = d->branch_type;
    j.dgate = q.shared_gate ? dgate : nullptr;
    j.rows = a.rows, j.gate_rows = a.gate_rows, j.rows_per_gate = a.rows_per_gate;
    j.teams = s.teams, j.hidden = a.hidden;
    dim3 grid((a.hidden + 31) / 32, (unsigned)std::min<uint64_t>(4 + (j.dgate ? a.gate_rows : 0), 4096));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(256), cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_norm_join, j);
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
