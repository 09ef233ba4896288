// ops_common.cuh -- what the training operators' translation units share: typed
// loads and stores, block reductions, and the host side's error reporting and
// launches.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <exception>
#include <mutex>
#include <string>
#include <utility>

#include "../../include/bf16opt.h"

// Records a handle-less call's message for bf16opt_last_error(NULL) and returns
// `code` (bf16opt.cu; not exported).
__attribute__((visibility("hidden"))) int bf16opt_fail_unbound(int code, const char *msg);

namespace bf16ops {

// ------------------------------------------------------------------ device side

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Largest of the warp's values (NaN passed over), in every lane.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// 2^x by the special-function unit, to two units in the last place (less than what the exponent's own product is
// rounded by, from |x| of a few on), subnormal results flushed to 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two FP32 numbers in one register pair: one instruction for both.
#define BF16OPS_PAIR_OP(name, op)                                                                                             \
    __device__ __forceinline__ float2 name(float2 a, float2 b) {                                                             \
        float2 r;                                                                                                            \
        asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n " op " r, a, b;\n mov.b64 {%0, %1}, r;\n}" \
            : "=f"(r.x), "=f"(r.y)                                                                                           \
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                                                       \
        return r;                                                                                                            \
    }
BF16OPS_PAIR_OP(add2, "add.rn.f32x2")
BF16OPS_PAIR_OP(mul2, "mul.rn.f32x2")
#undef BF16OPS_PAIR_OP
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n .reg .b64 a, b, c, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 r, a, b, c;\n mov.b64 {%0, %1}, r;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 16 bytes from global to shared memory without registers in between; the
// thread's copies up to a commit are one group.
__device__ __forceinline__ void copy_async16(void *smem, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of this thread's newest groups are in flight.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The same for a number that is the same in all threads; above 7 it waits for more than it need.
__device__ __forceinline__ void copy_wait_for(uint32_t n) {
    if (n == 0) copy_wait<0>();
    else if (n == 1) copy_wait<1>();
    else if (n == 2) copy_wait<2>();
    else if (n == 3) copy_wait<3>();
    else if (n == 4) copy_wait<4>();
    else if (n == 5) copy_wait<5>();
    else if (n == 6) copy_wait<6>();
    else copy_wait<7>();
}

constexpr float kLog2e = 1.44269504088896340736f;

// One 16-byte vector of the element type T: 8 bf16 or 4 FP32.
template <class T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void unpack(const uint4 &v, float (&f)[8]) {
        f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void unpack(const uint4 &v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float &d, float x) { d = x; }

// One element of a buffer whose type is known at run time (BF16OPT_TYPE_*).
__device__ __forceinline__ float load_typed(const void *p, int type, uint64_t i) {
    return type == BF16OPT_TYPE_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i])
                                     : reinterpret_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_typed(void *p, int type, uint64_t i, float x) {
    if (type == BF16OPT_TYPE_BF16) reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else reinterpret_cast<float *>(p)[i] = x;
}
__device__ __forceinline__ int64_t load_index(const void *p, int type, uint64_t i) {
    return type == BF16OPT_INDEX_I32 ? (int64_t)reinterpret_cast<const int32_t *>(p)[i]
                                     : reinterpret_cast<const int64_t *>(p)[i];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Rows [team_row(p), team_row(p + 1)) of `rows` are team p's: floor(p rows / teams).
__host__ __device__ inline uint64_t team_row(uint64_t rows, uint32_t teams, uint32_t p) {
    return rows / teams * p + rows % teams * p / teams;
}
// The team of a row: the last p with p rows / teams < row + 1.  (rows < 2^40)
__device__ __forceinline__ uint32_t team_of(uint64_t rows, uint32_t teams, uint64_t row) {
    return (uint32_t)(((row + 1) * teams - 1) / rows);
}

// Programmatic dependent launch: pdl_enter waits for the prerequisite grids
// before the first memory access; pdl_leave, at a CTA's end, lets the successor's CTAs be
// scheduled once every CTA has come that far.  (Allowed at the start,
// they take the slots that come free first: a successor of one or two CTAs per SM
// then sits on part of the SMs.  The router's two passes over 262144 x 256 took
// 741 us back to back that way, 533 us one at a time.)
__device__ __forceinline__ void pdl_enter() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_leave() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// -------------------------------------------------------------------- host side

inline int fail(int code, const std::string &msg) { return bf16opt_fail_unbound(code, msg.c_str()); }
inline int fail_cuda(cudaError_t e, const char *what) {
    return fail(BF16OPT_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

inline bool type_ok(int t) { return t == BF16OPT_TYPE_BF16 || t == BF16OPT_TYPE_F32; }
inline bool index_ok(int t) { return t == BF16OPT_INDEX_I32 || t == BF16OPT_INDEX_I64; }
inline uint64_t type_bytes(int t) { return t == BF16OPT_TYPE_BF16 ? 2 : 4; }
inline uint64_t index_bytes(int t) { return t == BF16OPT_INDEX_I32 ? 4 : 8; }
inline bool misaligned(const void *p, uint64_t bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

// Rows of `len` elements, `stride` apart: the bytes they span (0 for no rows).
// false if that does not fit 63 bits.
inline bool span_bytes(uint64_t rows, uint64_t stride, uint64_t len, uint64_t elem, uint64_t &out) {
    const unsigned __int128 n = rows == 0 ? 0 : ((unsigned __int128)(rows - 1) * stride + len) * elem;
    out = (uint64_t)n;
    return n < ((unsigned __int128)1 << 63);
}
inline bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}

// Multiprocessors of the current device; 0 without one.  Asked once per device.
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < 64)
        if (const int n = known[dev].load(std::memory_order_relaxed)) return n;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// An exception (an allocation of a message's string) does not cross the C ABI.
template <class F>
int guarded(F &&f) {
    try {
        return f();
    } catch (const std::exception &) {
        return bf16opt_fail_unbound(BF16OPT_ERR_OOM, "host allocation failed");
    }
}

struct Launch {
    unsigned grid, block;
    size_t smem = 0;
    cudaStream_t stream = nullptr;
    unsigned cluster = 0;    // CTAs per cluster; 0: no cluster
    bool dependent = false;  // programmatic dependent launch (the kernel calls pdl_enter)
};

constexpr size_t kMaxDynamic = 220 * 1024;   // shared memory that a kernel may ask for at a launch

// Clusters (or CTAs) of this launch that the device holds at once, with the kernel
// allowed its shared memory.  Both questions cost microseconds, so the answers
// are kept, by kernel, device and shape.
template <class... KArgs>
cudaError_t clusters_that_fit(const Launch &l, void (*kernel)(KArgs...), int &n, bool ask = false) {
    struct Known {
        const void *kernel;
        int device;
        unsigned cluster, block;
        size_t smem;
        int n;
    };
    static std::mutex mu;
    static Known known[64];
    static unsigned used = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const void *key = reinterpret_cast<const void *>(kernel);
    std::lock_guard<std::mutex> lock(mu);
    if (!ask)
        for (unsigned i = 0; i < std::min(used, 64u); ++i) {
            const Known &k = known[i];
            if (k.kernel == key && k.device == dev && k.cluster == l.cluster && k.block == l.block && k.smem == l.smem) {
                n = k.n;
                return cudaSuccess;
            }
        }
    if (l.smem > 32 * 1024) {   // with the static arrays, more than a kernel may have unasked
        // as much as any shape of it takes, so that a smaller one's answer does not take it back
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDynamic);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.cluster);
    cfg.blockDim = dim3(l.block);
    cfg.dynamicSmemBytes = l.smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = l.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e == cudaSuccess && n < 1) e = cudaErrorLaunchOutOfResources;
    if (e == cudaSuccess) known[used++ % 64] = Known{key, dev, l.cluster, l.block, l.smem, n};
    return e;
}

template <class... KArgs, class... Args>
cudaError_t launch(const Launch &l, void (*kernel)(KArgs...), const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.grid);
    cfg.blockDim = dim3(l.block);
    cfg.dynamicSmemBytes = l.smem;
    cfg.stream = l.stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (l.cluster) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = l.cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (l.dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaErrorInvalidValue && l.smem > 32 * 1024) {   // a context that replaced a reset one has the kernel without its shared memory
        cudaGetLastError();
        int fit = 0;
        e = clusters_that_fit(l, kernel, fit, true);
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, args...);
    }
    return e;
}

}  // namespace bf16ops
