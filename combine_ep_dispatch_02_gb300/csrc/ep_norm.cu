// ep_norm.cu -- RMS norm with the residual's addition and an e4m3 output with block scales: the
// step that makes the rows an FP8 dispatch takes.
//
// Per row of H elements, in FP32:
//   h = x + residual                          (written back rounded to the 16-bit type)
//   y = h * 1/sqrt(mean(h^2) + eps) * weight   (optionally written rounded, for the router)
//   per 128 elements: scale = max|y| / 448, code = e4m3(y / scale)
// The norm takes the unrounded h, so each output is rounded exactly once.
//
// HBM-bound: about 25 FP32 operations per element against 3 to 9 bytes.  A row is read once and
// stays in registers between the sum of squares and the outputs.  Lanes own 16-byte vectors, so
// the 16 lanes of half a warp hold one 128-element block and its maximum takes four shuffles.  Rows up
// to 1024 elements are one warp's, without a barrier; longer ones a CTA's, four vectors to a thread, so
// that several rows are in flight on an SM while one waits for its sum.
//
// 32768 rows of 7168 BF16 with residual and both outputs: 305 us, 6.95 TB/s (1.03 of the measured copy).
// One row: 3.8 us, the launch and one trip to memory and back.
#include "ep_layer.cuh"

namespace ep {
namespace {

struct NormArgs {
    const uint8_t* x;
    const uint8_t* residual;
    const void* weight;
    uint8_t* q;
    float* scales;
    uint8_t* h;
    uint8_t* y;
    int64_t rows, x_pitch, r_pitch;   // pitches in bytes
    int hidden, vecs, blocks;         // 16-byte vectors and 128-element blocks of a row
    int weight_fp32;
    float eps;
};

constexpr int kNormWarpsPerCta = 4;   // rows of a CTA when a row is one warp's
constexpr int kNormMaxThreads = 512;  // of a row's CTA: 128 registers each hold 8 vectors as floats
constexpr int kNormMaxHidden = kNormMaxThreads * 8 * 8;

// A row by one warp (WARP) or by the whole CTA; VPT vectors per thread.
template <bool FP16, bool WARP, int VPT>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarpsPerCta : kNormMaxThreads) ep_norm_kernel(const NormArgs a)
{
    const int lane = threadIdx.x & 31;
    const int t = WARP ? lane : threadIdx.x;
    const int stride = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * kNormWarpsPerCta + (threadIdx.x >> 5) : blockIdx.x;
    follow_predecessor();
    if (WARP && row >= a.rows) return;
    const uint8_t* x = a.x + row * a.x_pitch;
    float f[VPT][8];
    {
        uint4 vx[VPT], vr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * stride + t;
            vx[i] = make_uint4(0, 0, 0, 0);
            vr[i] = make_uint4(0, 0, 0, 0);
            if (v < a.vecs) {
                vx[i] = *reinterpret_cast<const uint4*>(x + 16 * (int64_t)v);
                if (a.residual) vr[i] = *reinterpret_cast<const uint4*>(a.residual + row * a.r_pitch + 16 * (int64_t)v);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            unpack8<FP16>(vx[i], f[i]);
            if (a.residual) {
                float r[8];
                unpack8<FP16>(vr[i], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] += r[j];
            }
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
        const int v = i * stride + t;
        if (a.h && v < a.vecs)
            *reinterpret_cast<uint4*>(a.h + (row * a.vecs + v) * 16) = pack8<FP16>(f[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (!WARP) {
        __shared__ float part[32];
        if (lane == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const float rstd = __frsqrt_rn(__fdiv_rn(sum, (float)a.hidden) + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * stride + t;
        const bool in = v < a.vecs;
        float w[8] = {};
        if (in) {
            if (a.weight_fp32) {
                const float4* wp = reinterpret_cast<const float4*>(a.weight) + 2 * v;
                const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
                w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
                w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
            } else {
                unpack8<FP16>(__ldg(reinterpret_cast<const uint4*>(a.weight) + v), w);
            }
        }
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[i][j] = f[i][j] * rstd * w[j];
            m = fmaxf(m, in ? fabsf(f[i][j]) : 0.0f);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float scale = e4m3_block_scale(m);
        const float inv = __frcp_rn(scale);
        if (in) {
            const uint2 q = make_uint2(e4m3x4_scaled(f[i][0], f[i][1], f[i][2], f[i][3], scale, inv),
                                       e4m3x4_scaled(f[i][4], f[i][5], f[i][6], f[i][7], scale, inv));
            *reinterpret_cast<uint2*>(a.q + (row * a.vecs + v) * 8) = q;
            if ((v & 15) == 0) a.scales[row * a.blocks + (v >> 4)] = scale;
            if (a.y) *reinterpret_cast<uint4*>(a.y + (row * a.vecs + v) * 16) = pack8<FP16>(f[i]);
        }
    }
}

template <bool FP16, bool WARP>
cudaError_t launch_norm(const NormArgs& a, int vpt, int threads, cudaStream_t s)
{
    const unsigned grid = (unsigned)(WARP ? (a.rows + kNormWarpsPerCta - 1) / kNormWarpsPerCta : a.rows);
    switch (vpt) {
    case 1: return launch_dependent(ep_norm_kernel<FP16, WARP, 1>, dim3(grid), dim3(threads), 0, s, a);
    case 2: return launch_dependent(ep_norm_kernel<FP16, WARP, 2>, dim3(grid), dim3(threads), 0, s, a);
    case 4: return launch_dependent(ep_norm_kernel<FP16, WARP, 4>, dim3(grid), dim3(threads), 0, s, a);
    default: return launch_dependent(ep_norm_kernel<FP16, WARP, 8>, dim3(grid), dim3(threads), 0, s, a);
    }
}

}  // namespace
}  // namespace ep

extern "C" int ep_rms_norm_fp8(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                               const void* weight, int weight_fp32, int dtype, int64_t rows, int hidden,
                               float eps, void* q, float* scales, void* h, void* y, void* stream)
{
    using namespace ep;
    if (dtype != EP_BF16 && dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: dtype=%d is neither EP_BF16 nor EP_FP16", dtype);
    if (hidden < 16 || hidden > kNormMaxHidden || hidden % 16 != 0)
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: hidden=%d is not a multiple of 16 in 16..%d", hidden,
                          kNormMaxHidden);
    if (rows < 0 || rows >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: rows=%lld outside 0..2^31-1", (long long)rows);
    if (!(eps >= 0.0f)) return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: eps=%g is negative or NaN", (double)eps);
    if (rows == 0) return EP_OK;
    if (!layer_aligned(x, 16) || x_stride < hidden || x_stride % 8 != 0)
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: x is NULL, not 16-byte aligned, or its row stride %lld is below "
                          "hidden or not a multiple of 8",
                          (long long)x_stride);
    if (residual && (!layer_aligned(residual, 16) || residual_stride < hidden || residual_stride % 8 != 0))
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: residual is not 16-byte aligned, or its row stride %lld is below "
                          "hidden or not a multiple of 8",
                          (long long)residual_stride);
    if (!layer_aligned(weight, 16)) return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: weight is NULL or not 16-byte aligned");
    if (!layer_aligned(q, 16) || !layer_aligned(scales, 4))
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: q or scales is NULL or misaligned");
    if ((h && !layer_aligned(h, 16)) || (y && !layer_aligned(y, 16)))
        return layer_fail(EP_ERR_ARG, "ep_rms_norm_fp8: h or y is not 16-byte aligned");
    NormArgs a{};
    a.x = (const uint8_t*)x; a.residual = (const uint8_t*)residual; a.weight = weight;
    a.q = (uint8_t*)q; a.scales = scales; a.h = (uint8_t*)h; a.y = (uint8_t*)y;
    a.rows = rows; a.x_pitch = 2 * x_stride; a.r_pitch = 2 * residual_stride;
    a.hidden = hidden; a.vecs = hidden / 8; a.blocks = (hidden + 127) / 128;
    a.weight_fp32 = weight_fp32; a.eps = eps;
    const bool fp16 = dtype == EP_FP16;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (a.vecs <= 128) {   // a row per warp
        const int vpt = a.vecs <= 32 ? 1 : a.vecs <= 64 ? 2 : 4;
        e = fp16 ? launch_norm<true, true>(a, vpt, 32 * kNormWarpsPerCta, s)
                 : launch_norm<false, true>(a, vpt, 32 * kNormWarpsPerCta, s);
    } else {
        const int vpt = a.vecs <= 4 * kNormMaxThreads ? 4 : 8;
        const int threads = ((a.vecs + vpt - 1) / vpt + 31) / 32 * 32;
        e = fp16 ? launch_norm<true, false>(a, vpt, threads, s) : launch_norm<false, false>(a, vpt, threads, s);
    }
    return layer_cuda(e, "ep_rms_norm_fp8: launch");
}
