// ep_matmul.cu -- e4m3 matrix product with FP32 block scales, dense or by expert.
//
//   out[i][n] = sum over 128-blocks kb of  as[i][kb] * bs[g][n/128][kb] * sum_{k in kb} a[i][k] b[g][n][k]
//
// for the rows i of group g (offsets[g] .. offsets[g+1]), summed in FP32 and rounded once; or, with
// b holding gate rows and then up rows, z = gate * sigmoid(gate) * up in FP32, written as e4m3
// codes with one FP32 scale per 128 columns.
//
// Products of e4m3 values are exact in FP32, so the block sums keep FP32 accuracy and the scales
// enter once per block.
#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kMaxMatmulGroups = 4096;

struct MatmulArgs {
    const uint8_t* a;
    const float* as;
    const uint8_t* b;
    const float* bs;
    const int32_t* offsets;   // [groups + 1], or NULL: one group of all rows
    void* out;
    float* out_scales;
    int* status;
    int64_t rows;
    int groups, N, K, kb;     // N: output columns of a row (swiglu: half the rows of b)
    int nb;                   // 128-row blocks of b in one group
    int swiglu, dtype;
};

// First and last row of group g, clamped to the buffer.
__device__ __forceinline__ void group_rows(const MatmulArgs& p, int g, int& lo, int& hi)
{
    if (!p.offsets) { lo = 0; hi = (int)p.rows; return; }
    lo = max(0, min(p.offsets[g], (int)p.rows));
    hi = max(lo, min(p.offsets[g + 1], (int)p.rows));
}

constexpr int kTileM = 32, kTileN = 128, kTileK = 32, kThreads = 256;

__device__ __forceinline__ float2 codes2(uint32_t c) { return e4m3x2_to_float2(c & 0xFFFFu); }

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads) ep_matmul_kernel(const MatmulArgs p)
{
    constexpr int kHalves = SWIGLU ? 2 : 1;
    __shared__ float sa[kTileK][kTileM + 1];
    __shared__ float sb[kHalves][kTileK][kTileN + 1];
    __shared__ int found[3];
    if (threadIdx.x == 0) {   // the row tile this CTA takes
        int t = blockIdx.x;
        found[0] = -1;
        for (int g = 0; g < p.groups; ++g) {
            int lo, hi;
            group_rows(p, g, lo, hi);
            const int n = (hi - lo + kTileM - 1) / kTileM;
            if (t < n) {
                found[0] = g;
                found[1] = lo + t * kTileM;
                found[2] = hi;
                break;
            }
            t -= n;
        }
    }
    __syncthreads();
    const int g = found[0], m0 = found[1], m1 = found[2];
    if (g < 0) return;
    const int n0 = blockIdx.y * kTileN;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;   // 4 rows x (4 columns, 32 apart)
    const int64_t bn = SWIGLU ? 2 * (int64_t)p.N : p.N;
    float acc[kHalves][4][4] = {}, blk[kHalves][4][4] = {};
    for (int k0 = 0; k0 < p.kb * 128; k0 += kTileK) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTileM * kTileK / 2; i += kThreads) {
            const int r = i / (kTileK / 2), k = i % (kTileK / 2) * 2;
            float2 v = make_float2(0.0f, 0.0f);
            if (m0 + r < m1 && k0 + k < p.K)
                v = codes2(*reinterpret_cast<const uint16_t*>(p.a + (int64_t)(m0 + r) * p.K + k0 + k));
            sa[k][r] = v.x;
            sa[k + 1][r] = v.y;
        }
        for (int i = threadIdx.x; i < kHalves * kTileN * kTileK / 2; i += kThreads) {
            const int h = i / (kTileN * kTileK / 2), j = i % (kTileN * kTileK / 2);
            const int n = j / (kTileK / 2), k = j % (kTileK / 2) * 2;
            float2 v = make_float2(0.0f, 0.0f);
            if (n0 + n < p.N && k0 + k < p.K)
                v = codes2(*reinterpret_cast<const uint16_t*>(p.b + (g * bn + (int64_t)h * p.N + n0 + n) * p.K + k0 + k));
            sb[h][k][n] = v.x;
            sb[h][k + 1][n] = v.y;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTileK; ++k) {
            float av[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) av[i] = sa[k][4 * ty + i];
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float bv = sb[h][k][tx + 32 * j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) blk[h][i][j] = fmaf(av[i], bv, blk[h][i][j]);
                }
        }
        if ((k0 + kTileK) % 128 == 0) {
            const int kb = k0 / 128;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = min(m0 + 4 * ty + i, m1 - 1);
                    const float s = p.as[(int64_t)m * p.kb + kb];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t row = min(n0 + tx + 32 * j, p.N - 1) + (int64_t)h * p.N;
                        const float bs = p.bs[(g * (int64_t)p.nb + row / 128) * p.kb + kb];
                        acc[h][i][j] = fmaf(blk[h][i][j], s * bs, acc[h][i][j]);
                        blk[h][i][j] = 0.0f;
                    }
                }
        }
    }
    if constexpr (!SWIGLU) {
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + 4 * ty + i, n = n0 + tx + 32 * j;
                if (m >= m1 || n >= p.N) continue;
                const int64_t at = (int64_t)m * p.N + n;
                if (p.dtype == EP_FP16) ((__half*)p.out)[at] = __float2half_rn(acc[0][i][j]);
                else ((__nv_bfloat16*)p.out)[at] = __float2bfloat16_rn(acc[0][i][j]);
            }
    } else {
        float z[4][4];
        for (int i = 0; i < 4; ++i) {
            float m = 0.0f;
            for (int j = 0; j < 4; ++j) {
                const float gate = acc[0][i][j];
                z[i][j] = gate / (1.0f + expf(-gate)) * acc[1][i][j];
                if (n0 + tx + 32 * j < p.N) m = fmaxf(m, fabsf(z[i][j]));
            }
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float scale = e4m3_block_scale(m);
            const int row = m0 + 4 * ty + i;
            if (row >= m1) continue;
            if (tx == 0) p.out_scales[(int64_t)row * ((p.N + 127) / 128) + blockIdx.y] = scale;
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 32 * j;
                if (n < p.N) ((uint8_t*)p.out)[(int64_t)row * p.N + n] = (uint8_t)e4m3x2(__fdiv_rn(z[i][j], scale), 0.0f);
            }
        }
    }
}

}  // namespace
}  // namespace ep

extern "C" int ep_matmul_fp8(const void* a, const float* a_scales, const void* b, const float* b_scales,
                             const int32_t* offsets, int64_t rows, int groups, int columns, int inner, int swiglu,
                             int dtype, void* out, float* out_scales, int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_matmul_fp8";
    if (rows < 0 || rows >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: rows=%lld outside 0..2^31-1", who, (long long)rows);
    if (groups < 1 || groups > kMaxMatmulGroups || (!offsets && groups != 1))
        return layer_fail(EP_ERR_ARG, "%s: groups=%d outside 1..%d, or several without offsets", who, groups,
                          kMaxMatmulGroups);
    if (inner < 16 || inner % 16 != 0 || inner > 1 << 20)
        return layer_fail(EP_ERR_ARG, "%s: inner=%d is not a multiple of 16 in 16..2^20", who, inner);
    if (columns < 1 || columns > 1 << 20 || (swiglu && columns % 32 != 0))
        return layer_fail(EP_ERR_ARG, "%s: columns=%d outside 1..2^20, or not a multiple of 32 with SwiGLU", who,
                          columns);
    if ((int64_t)groups * columns >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: groups*columns=%d*%d reaches 2^31", who, groups, columns);
    if (swiglu ? dtype != EP_FP8_E4M3 : dtype != EP_BF16 && dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "%s: dtype=%d is not EP_BF16 or EP_FP16 (EP_FP8_E4M3 with SwiGLU)", who, dtype);
    if (!layer_aligned(device_status, 4))
        return layer_fail(EP_ERR_ARG, "%s: device_status is NULL or not 4-byte aligned", who);
    if (rows == 0) return EP_OK;
    if (!layer_aligned(a, 16) || !layer_aligned(b, 16) || !layer_aligned(a_scales, 4) || !layer_aligned(b_scales, 4))
        return layer_fail(EP_ERR_ARG, "%s: a, b or a scale array is NULL or misaligned", who);
    if (!layer_aligned(out, 16) || (swiglu && !layer_aligned(out_scales, 4)))
        return layer_fail(EP_ERR_ARG, "%s: out or out_scales is NULL or misaligned", who);
    if (offsets && !layer_aligned(offsets, 4)) return layer_fail(EP_ERR_ARG, "%s: offsets is not 4-byte aligned", who);
    MatmulArgs p{};
    p.a = (const uint8_t*)a; p.as = a_scales; p.b = (const uint8_t*)b; p.bs = b_scales; p.offsets = offsets;
    p.out = out; p.out_scales = out_scales; p.status = device_status; p.rows = rows; p.groups = groups;
    p.K = inner; p.kb = (inner + 127) / 128; p.N = swiglu ? columns / 2 : columns; p.nb = (columns + 127) / 128;
    p.swiglu = swiglu; p.dtype = dtype;
    const dim3 grid((unsigned)(rows / kTileM + groups + 1), (unsigned)((p.N + kTileN - 1) / kTileN));
    cudaStream_t s = (cudaStream_t)stream;
    if (swiglu) ep_matmul_kernel<true><<<grid, kThreads, 0, s>>>(p);
    else ep_matmul_kernel<false><<<grid, kThreads, 0, s>>>(p);
    return layer_cuda(cudaGetLastError(), "ep_matmul_fp8: launch");
}
