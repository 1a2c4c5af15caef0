// zero_device.cuh -- what the device translation units share: the sharded step's device-resident state,
// element conversions, the AdamW rule, fixed-order sums, bounded mbarrier waits, and a few host helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <string>
#include <utility>

#include "zero_internal.h"

namespace zero {
namespace {

// ------------------------------------------------------------------ host helpers

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

inline int device_sms(int dev)
{
    static std::mutex mu;
    static int cache[64] = {0};
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64) return 0;
    if (cache[dev] == 0) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev] = sms;
    }
    return cache[dev];
}

inline zero_status_t cuda_fail(cudaError_t e, const char* what)
{
    return fail(ZERO_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Allow a kernel `bytes` of dynamic shared memory (beyond 48 KB that takes a call) on the current
// device, once a kernel and device.
template <auto KERNEL>
inline cudaError_t allow_shared(int bytes)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// Launch a kernel that begins with after_earlier_work(): its blocks may be set up while the kernel before
// it on the stream still runs (programmatic dependent launch), which hides most of a launch's latency: a step
// over small tensors (two launches) 14.3 -> 10.0 us, one token's linear layer 16.4 -> 13.7, small gradients of
// four launches 53.5 -> 49.4.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters_after(void (*kernel)(KArgs...), dim3 cluster, dim3 grid, dim3 threads, size_t shared, cudaStream_t s, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster.x;
    attrs[1].val.clusterDim.y = cluster.y;
    attrs[1].val.clusterDim.z = cluster.z;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same without clusters, or with those that the kernel's __cluster_dims__ gives it.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 threads, size_t shared, cudaStream_t s, Args&&... args)
{
    return launch_clusters_after(kernel, dim3(1), grid, threads, shared, s, std::forward<Args>(args)...);
}

// In every kernel that launch_after starts, by every thread, before any access to global memory: every earlier
// kernel of the stream has ended and its writes are seen (PTX promises that to a kernel that waits itself, and
// to no other); then the next launch may be set up once every block is here.
__device__ __forceinline__ void after_earlier_work()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Read and clear a kernel's error word (on a device variable), after the work on `s`.
template <typename W>
inline cudaError_t take_error_word(W& symbol, uint32_t* word, cudaStream_t s)
{
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, symbol, sizeof(*word), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *word == 0) return e;
    const uint32_t none = 0;
    e = cudaMemcpyToSymbolAsync(symbol, &none, sizeof(none), 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

// ------------------------------------------------------------------ device-resident step state

// First 96 bytes of the workspace.  Written by the commit (the last re-cast block or
// commit_kernel), by the host before the first step, and by the kernels' atomics (flag,
// error, norm tickets); read by the step and re-cast kernels of the following step.
struct DevState {
    uint32_t flag;          // OR of the non-finite flags of the open step
    uint32_t cur;           // current half of every ping-pong pair
    uint32_t last_skipped;  // 1 if the last finished step was skipped
    uint32_t blocks_done;   // blocks of the running norm launch that have stored their partial
    int64_t t;              // applied steps
    int64_t skipped;        // skipped steps, total
    int64_t good;           // applied steps since the last change of the loss scale
    int64_t finished;       // finished steps (applied + skipped)
    double scale;           // loss scale of the next step
    double norm2;           // open step: sum of fp32(g*g) so far
    double last_norm2;      // last finished step's sum
    uint32_t norm_valid;    // open step computed a norm
    uint32_t last_norm_valid;
    uint32_t error;         // bit 0: a barrier wait of the staged step ran out; bit 1: a drain
                            // ran out; bit 2: a barrier wait of the staged gather ran out; bit 3: a
                            // wait of another optimizer's part of the step ran out
                            // (sticky until read; every step finished meanwhile is discarded)
    uint32_t pad32;
    int64_t pad;
};
static_assert(sizeof(DevState) == 96, "DevState layout");

static_assert(sizeof(DevState) <= kStateBytes, "DevState fits its workspace slot");

// ------------------------------------------------------------------ element helpers

// 16-bit -> fp32 widening (exact).  bf16 is the upper half of an IEEE binary32.
template <int DT>
__device__ __forceinline__ float widen1(uint16_t h)
{
    if constexpr (DT == ZERO_BF16) return __uint_as_float((uint32_t)h << 16);
    else return __half2float(__ushort_as_half(h));
}

template <int DT>
__device__ __forceinline__ void widen2(uint32_t w, float& lo, float& hi)
{
    if constexpr (DT == ZERO_BF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    } else {
        __half2 h = *reinterpret_cast<const __half2*>(&w);
        float2 f = __half22float2(h);
        lo = f.x;
        hi = f.y;
    }
}

// fp32 -> 16-bit, round to nearest even.
template <int DT>
__device__ __forceinline__ uint16_t narrow1(float f)
{
    if constexpr (DT == ZERO_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    else return __half_as_ushort(__float2half_rn(f));
}

template <int DT>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    if constexpr (DT == ZERO_BF16) {
        __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

__device__ __forceinline__ bool nonfinite(float g)
{
    return (__float_as_uint(g) & 0x7F800000u) == 0x7F800000u;
}

// Two floats in one 64-bit register: one instruction rounds both, each as by itself.
struct F2 {
    unsigned long long v;
};

__device__ __forceinline__ F2 pair(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ F2 both(float a) { return pair(a, a); }

__device__ __forceinline__ void split(F2 p, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}

__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// a + b with a kept a rounded product: `one` is 1 from memory, unknown to the compiler, which would
// contract the packed product and sum to one rounding.
__device__ __forceinline__ F2 add_apart(F2 a, F2 b, F2 one)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(one.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The constants that depend on t, the loss scale and the gradient norm, formed per block.
struct StepK {
    float step;   // lr / (1 - beta1^t)
    float bc2s;   // sqrt(1 - beta2^t)
    float inv;    // 1 / (N_d * loss_scale)
    float coef;   // clip mode: min(1, max_norm / (norm + 1e-6)); else 1
};

// Per-thread sum of the fp32 squares as an unevaluated pair hi + lo of floats, extended by an
// error-free TwoSum (Knuth) per term: ~48 significant bits from fp32 operations only (GB300's
// fp64 rate is far below its fp32 rate).  Converted to double once, at the end of the thread.
struct NormAcc {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float p)
    {
        const float s = __fadd_rn(hi, p);
        const float bp = __fsub_rn(s, hi);
        const float ap = __fsub_rn(s, bp);
        const float e = __fadd_rn(__fsub_rn(hi, ap), __fsub_rn(p, bp));
        hi = s;
        lo = __fadd_rn(lo, e);
    }
    // beyond the range hi is infinite and lo not a number
    __device__ __forceinline__ double value() const { return isinf(hi) ? (double)hi : (double)hi + (double)lo; }
};

// AdamW on one element with separately rounded IEEE operations (no contraction):
//   m = b1 m + (1-b1) g ; v = b2 v + (1-b2) g^2 ; d = sqrt(v)/sqrt(bc2) + eps
//   p = p - (lr wd) p   ; p = p - (lr/bc1) (m / d)
// k[0..5] (b1, 1-b1, b2, 1-b2, eps, lr*wd) stay in the kernel parameters.
__device__ __forceinline__ void adamw1(float g, float& p, float& m, float& v, const float* k,
                                       const StepK& sk)
{
    m = __fadd_rn(__fmul_rn(k[0], m), __fmul_rn(k[1], g));
    v = __fadd_rn(__fmul_rn(k[2], v), __fmul_rn(k[3], __fmul_rn(g, g)));
    const float d = __fadd_rn(__fdiv_rn(__fsqrt_rn(v), sk.bc2s), k[4]);
    p = __fsub_rn(p, __fmul_rn(k[5], p));
    p = __fsub_rn(p, __fmul_rn(sk.step, __fdiv_rn(m, d)));
}

__device__ __forceinline__ uint4 ld_stream(const void* p)
{
    return __ldcs(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ uint2 ld_stream8(const void* p)
{
    return __ldcs(reinterpret_cast<const uint2*>(p));
}

// Sum of one double over a block of NT threads in a fixed pattern (shuffle tree per warp,
// warps in order); the result is valid in thread 0.
template <int NT>
__device__ __forceinline__ double block_sum_fixed(double x, double* warp_sum)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_down_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    double b = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < NT / 32; ++w) b += warp_sum[w];
    __syncthreads();
    return b;
}

// ------------------------------------------------------------------ bounded barrier waits

constexpr uint32_t kWaitIterCap = 1u << 26;              // polls per wait, whatever the clock

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Non-blocking probe of the same condition.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait until the phase of parity `parity` of barrier `bar` has completed.  False when
// limit_ns of %globaltimer (or kWaitIterCap polls) pass first; limit 0 gives up as soon as
// the first, non-blocking probe fails.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    if (mbar_test(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < kWaitIterCap; ++i) {
        if (global_ns() - t0 >= limit_ns) return false;
        if (mbar_try(bar, parity)) return true;
    }
    return false;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

}  // namespace
}  // namespace zero
