// ep_layer.cuh -- declarations shared by the expert-layer operators (norm, sort by expert and
// return, block-scaled FP8 product): host-side argument checks and 16-bit vector arithmetic.
//
// These operators hold no state of their own: every buffer is the caller's, every condition the
// host can check fails with a message before any launch, and what only the device can see is
// recorded in the caller's status word.
#pragma once

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ep_common.cuh"

namespace ep {

int record_error(int code, const char* msg);   // sets the message read by ep_last_error()

inline int layer_fail(int code, const char* fmt, ...)
{
    char msg[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return record_error(code, msg);
}

inline int layer_cuda(cudaError_t e, const char* who)
{
    if (e == cudaSuccess) return EP_OK;
    cudaGetLastError();   // reported here: not once more to the next caller that asks the runtime
    return layer_fail(EP_ERR_CUDA, "%s: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool layer_aligned(const void* p, size_t a) { return p != nullptr && ((uintptr_t)p % a) == 0; }

// SMs of the current device, 0 if it cannot be told (looked up once per device)
inline int layer_num_sms()
{
    static std::atomic<int> sms[64] = {};
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n != 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    sms[dev].store(n, std::memory_order_relaxed);
    return n;
}

#ifdef __CUDACC__

// Lets launches of K take all the shared memory a CTA can have.  The limit is one per kernel and device, and
// host threads share it: it is raised once to the most there is, never to one call's size, which another
// thread's smaller call could lower again before the launch.  Two threads may both raise it, to the same value.
template <auto* K>
cudaError_t allow_all_shared()
{
    static std::atomic<uint64_t> raised{0};   // a bit per device
    int dev = -1, most = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (raised.load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, K);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)f.sharedSizeBytes);
    if (e == cudaSuccess) raised.fetch_or(bit, std::memory_order_release);
    return e;
}

// Every kernel of these operators is launched as a programmatic dependent (launch_dependent), whatever
// precedes it on the stream, and starts with this: its launch and set-up overlap the tail of the kernel
// before it, it touches no memory before that kernel has completed, and only then lets its own
// dependent be scheduled.  In a stream of small calls that hides 1 to 2 us of each.
__device__ __forceinline__ void follow_predecessor()
{
    wait_for_predecessor();
    allow_dependents();
}

// Eight 16-bit values of a 16-byte vector as floats, and back (rounded to nearest even once).
template <bool FP16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FP16) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        } else {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (FP16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
}

template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack2<FP16>(f[0], f[1]), pack2<FP16>(f[2], f[3]), pack2<FP16>(f[4], f[5]),
                      pack2<FP16>(f[6], f[7]));
}

// FP32 scale of a 128-element block with largest magnitude m, as the quantising dispatch defines
// it: m / 448, and 1 for a block of zeros (fmaxf drops NaN, so a block of NaN also gets 1).
__device__ __forceinline__ float e4m3_block_scale(float m) { return m > 0.0f ? __fdiv_rn(m, 448.0f) : 1.0f; }

// Four e4m3 codes of v / scale; inv = RN(1 / scale).  The correctly rounded quotient comes from
// the reciprocal and one residual step where no intermediate underflows or overflows (see
// div_by_scale), from an IEEE division elsewhere; the branch is uniform over a block's lanes.
__device__ __forceinline__ uint32_t e4m3x4_scaled(float a, float b, float c, float d, float scale, float inv)
{
    if (scale >= 0x1p-60f && scale <= 0x1p100f)
        return e4m3x2(div_by_scale(a, scale, inv), div_by_scale(b, scale, inv)) |
               (e4m3x2(div_by_scale(c, scale, inv), div_by_scale(d, scale, inv)) << 16);
    return e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)) |
           (e4m3x2(__fdiv_rn(c, scale), __fdiv_rn(d, scale)) << 16);
}

// The same by a multiplication with the reciprocal, for values that are themselves off by more than the
// half unit in the last place that this may add; by a division where the reciprocal would be too large.
__device__ __forceinline__ float near_quotient(float v, float scale, float inv)
{
    return scale >= 0x1p-100f ? v * inv : __fdiv_rn(v, scale);
}

__device__ __forceinline__ uint32_t e4m3x4_near(float a, float b, float c, float d, float scale, float inv)
{
    if (scale >= 0x1p-100f) return e4m3x2(a * inv, b * inv) | (e4m3x2(c * inv, d * inv) << 16);
    return e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale)) |
           (e4m3x2(__fdiv_rn(c, scale), __fdiv_rn(d, scale)) << 16);
}

#endif  // __CUDACC__

}  // namespace ep
