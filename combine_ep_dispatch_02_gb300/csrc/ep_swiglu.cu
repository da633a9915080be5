// ep_swiglu.cu -- SwiGLU for training: its input is kept in 8 bits, and its gradient is taken from there.
//
//   forward, per row of [gate | up]:  z = gate * sigmoid(gate) * up, written as e4m3 codes with one FP32 scale per
//                                     128 columns; gate and up themselves as codes with a scale per 128 columns of
//                                     the row of both
//   backward, from those codes:       s = sigmoid(gate);  dgate = dz * up * s * (1 + gate * (1 - s)),
//                                     dup = dz * gate * s, in 16 bits and, if asked, as codes with scales too
//
// HBM-bound by its bytes (7 of a z forward, 8 or 10 backward), with arithmetic close behind: a lane owns 8
// columns of gate and the same 8 of up, so sixteen lanes hold a block of 128, its maximum takes four shuffles and nothing
// passes through shared memory.  32768 rows of 2048 take 84 us (5.6 TB/s), the gradient with codes 103 us (6.6 TB/s): the
// forward pass has three quantisers and a sigmoid for 7 bytes, and its instructions take as long as its bytes.  Where the
// row's blocks straddle gate and up (inner no multiple of 128), blocks of the row are quantised by sixteen lanes of their own,
// which read again what their neighbours have just read and, in the gradient, compute it again: 32768 rows of 2064 take 159 us,
// the gradient with codes 162.
#include "ep_layer.cuh"

namespace ep {
namespace {

// Small CTAs, nine to an SM, whose ends lie apart: 32768 rows of 2048 84.4 us and, the gradient, 103.2; with 256 threads 88.1
// and 108.4, with ten CTAs (51 registers) 87.5 and 102.8, with 512 threads 96 and 115.
constexpr int kSwigluThreads = 128, kSwigluCtas = 9;
constexpr int kSwigluTeams = kSwigluThreads / 16;   // half warps, a block of 128 columns each
constexpr int kSwigluUnits = 2;                     // blocks of a half warp, so that both loads are on their way at once

struct SwigluArgs {
    const uint8_t* x;           // gate | up (forward) or dz (backward), 16-bit
    const uint8_t* saved_in;    // backward: codes of gate | up
    const float* saved_in_scales;
    const int32_t* end;         // rows at or past *end are left alone; may be NULL
    uint8_t* q;                 // codes of z (forward) or of the gradient (backward, may be NULL)
    float* scales;
    uint8_t* saved;             // forward: codes of gate | up
    float* saved_scales;
    uint8_t* d;                 // backward: gradient of gate | up, 16-bit
    int64_t pitch;              // bytes between rows of x
    int rows, inner;
    int z_blocks, row_blocks;   // 128-column blocks of z, and of gate | up
    uint32_t per_row, divide;   // blocks that the kernel works on in a row; the multiplier and shift of a division by them
    int shift;
};

// Whole-number division of u < 2^31 by d: u * ceil(2^(31 + l) / d) / 2^(31 + l) with d <= 2^l is exact (T. Granlund,
// P. L. Montgomery, "Division by invariant integers using multiplication", PLDI 1994).
void set_per_row(SwigluArgs& a, int d)
{
    int l = 0;
    while (((int64_t)1 << l) < d) ++l;
    a.per_row = (uint32_t)d;
    a.divide = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
    a.shift = 31 + l;
}

__device__ __forceinline__ uint32_t row_of(const SwigluArgs& a, uint32_t u) { return (uint32_t)(((uint64_t)u * a.divide) >> a.shift); }

// Largest magnitude over the sixteen lanes of a half warp; NaN counts as 0.
__device__ __forceinline__ float block_top(const float (&f)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
    for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// The same for two vectors of eight 16-bit values at once, in packed arithmetic.
template <bool FP16>
__device__ __forceinline__ float2 block_tops(const uint4& a, const uint4& b)
{
    auto larger = [](uint32_t x, uint32_t y) {
        if constexpr (FP16) {
            const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
            return *reinterpret_cast<const uint32_t*>(&m);
        } else {
            const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
            return *reinterpret_cast<const uint32_t*>(&m);
        }
    };
    constexpr uint32_t kMagnitude = 0x7FFF7FFFu;
    const uint32_t p = larger(larger(a.x & kMagnitude, a.y & kMagnitude), larger(a.z & kMagnitude, a.w & kMagnitude));
    const uint32_t q = larger(larger(b.x & kMagnitude, b.y & kMagnitude), larger(b.z & kMagnitude, b.w & kMagnitude));
    uint32_t m = larger(__byte_perm(p, q, 0x5410), __byte_perm(p, q, 0x7632));   // a's in the low half, b's in the high
#pragma unroll
    for (int o = 8; o; o >>= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float2 top = FP16 ? __half22float2(*reinterpret_cast<const __half2*>(&m)) : make_float2(bf16_lo(m), bf16_hi(m));
    return make_float2(fmaxf(top.x, 0.0f), fmaxf(top.y, 0.0f));   // a block of what is not a number alone: 0
}

// Eight codes of a lane of a block whose largest magnitude is `top` and, by the block's first lane, its scale.  The codes are
// those of the product with the scale's reciprocal, within three FP32 units of the quotient that they round.
__device__ __forceinline__ void write_codes(const float (&f)[8], float top, bool in, uint8_t* q, float* scale_out)
{
    if (!in) return;
    const float scale = quick_block_scale(top);
    uint2 codes;
    if (scale >= 0x1p-100f) {
        const float2 inv = both(quick_reciprocal(scale));
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = mul2(make_float2(f[2 * j], f[2 * j + 1]), inv);
            c[j] = e4m3x2(v.x, v.y);
        }
        codes = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    } else {
        codes = make_uint2(e4m3x4_near(f[0], f[1], f[2], f[3], scale, 0.0f), e4m3x4_near(f[4], f[5], f[6], f[7], scale, 0.0f));
    }
    *reinterpret_cast<uint2*>(q) = codes;
    if ((threadIdx.x & 15) == 0) *scale_out = scale;
}

// Eight codes times their scale.
__device__ __forceinline__ void read_codes(const uint2& c, float scale, float (&f)[8])
{
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = e4m3x2_to_float2(w[i]);
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

__device__ __forceinline__ int rows_in_use(const SwigluArgs& a)
{
    return a.end ? min(max(*a.end, 0), a.rows) : a.rows;
}

// Unit u: a block of z's columns with its gate and up, all three of which are quantised; with STRADDLE z alone, and the
// units past a row's z blocks quantise the row's own blocks.
template <bool FP16, bool STRADDLE>
__global__ void __launch_bounds__(kSwigluThreads, kSwigluCtas) ep_swiglu_saved_kernel(const SwigluArgs a)
{
    const int lane = threadIdx.x & 15;
    follow_predecessor();
    const int rows = rows_in_use(a);
    const uint32_t units = (uint32_t)rows * a.per_row;
    uint4 v[kSwigluUnits][2];
    int row[kSwigluUnits], block[kSwigluUnits];
#pragma unroll
    for (int i = 0; i < kSwigluUnits; ++i) {
        const uint32_t u = (blockIdx.x * kSwigluUnits + i) * kSwigluTeams + (threadIdx.x >> 4);
        const uint32_t r = row_of(a, u);
        row[i] = u < units ? (int)r : -1;
        block[i] = (int)(u - r * a.per_row);
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (row[i] < 0) continue;
        const uint8_t* x = a.x + row[i] * a.pitch;
        if (!STRADDLE || block[i] < a.z_blocks) {
            const int c = 128 * block[i] + 8 * lane;
            if (c < a.inner) {
                v[i][0] = *reinterpret_cast<const uint4*>(x + 2 * (int64_t)c);
                v[i][1] = *reinterpret_cast<const uint4*>(x + 2 * (int64_t)(a.inner + c));
            }
        } else {
            const int c = 128 * (block[i] - a.z_blocks) + 8 * lane;
            if (c < 2 * a.inner) v[i][0] = *reinterpret_cast<const uint4*>(x + 2 * (int64_t)c);
        }
    }
#pragma unroll
    for (int i = 0; i < kSwigluUnits; ++i) {
        // a warp's two units may be of different kinds, and the shuffles within are both's: one path for both
        const bool live = row[i] >= 0, own = STRADDLE && block[i] >= a.z_blocks;
        const int64_t r = max(row[i], 0);
        const int b = own ? block[i] - a.z_blocks : block[i], c = 128 * b + 8 * lane;
        float gate[8], up[8], z[8];
        unpack8<FP16>(v[i][0], gate);
        unpack8<FP16>(v[i][1], up);
        uint8_t* saved = a.saved + r * 2 * a.inner + c;
        float* saved_scales = a.saved_scales + r * a.row_blocks + b;
        if constexpr (!STRADDLE) {
            const float2 top = block_tops<FP16>(v[i][0], v[i][1]);
            write_codes(gate, top.x, live && c < a.inner, saved, saved_scales);
            write_codes(up, top.y, live && c < a.inner, saved + a.inner, saved_scales + a.z_blocks);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = own ? gate[j] : gate[j] * sigmoid_and_rest(gate[j]).x * up[j];
        write_codes(z, block_top(z), live && c < (own ? 2 : 1) * a.inner, own ? saved : a.q + r * a.inner + c,
                    own ? saved_scales : a.scales + r * a.z_blocks + b);
    }
}

// Unit u: a block of z's columns, whose gradients of gate and up leave; with QUANTISE also as codes.  With STRADDLE
// (and codes) a unit is instead a block of the row of both gradients.
template <bool FP16, bool QUANTISE, bool STRADDLE>
__global__ void __launch_bounds__(kSwigluThreads, kSwigluCtas) ep_swiglu_backward_kernel(const SwigluArgs a)
{
    const int lane = threadIdx.x & 15;
    follow_predecessor();
    const int rows = rows_in_use(a);
    const uint32_t units = (uint32_t)rows * a.per_row;
    uint2 g[kSwigluUnits], p[kSwigluUnits];
    uint4 dz[kSwigluUnits];
    float gs[kSwigluUnits], ps[kSwigluUnits];
    int row[kSwigluUnits], at[kSwigluUnits], col[kSwigluUnits];   // row, column of the gradients' row, column of z
#pragma unroll
    for (int i = 0; i < kSwigluUnits; ++i) {
        const uint32_t u = (blockIdx.x * kSwigluUnits + i) * kSwigluTeams + (threadIdx.x >> 4);
        const int r = (int)row_of(a, u);
        at[i] = 128 * (int)(u - r * a.per_row) + 8 * lane;
        row[i] = u < units && at[i] < (STRADDLE ? 2 : 1) * a.inner ? r : -1;
        col[i] = STRADDLE && at[i] >= a.inner ? at[i] - a.inner : at[i];
        g[i] = p[i] = make_uint2(0, 0);
        dz[i] = make_uint4(0, 0, 0, 0);
        gs[i] = ps[i] = 0.0f;
        if (row[i] < 0) continue;
        const uint8_t* codes = a.saved_in + (int64_t)r * 2 * a.inner;
        const float* s = a.saved_in_scales + (int64_t)r * a.row_blocks;
        g[i] = *reinterpret_cast<const uint2*>(codes + col[i]);
        p[i] = *reinterpret_cast<const uint2*>(codes + a.inner + col[i]);
        dz[i] = *reinterpret_cast<const uint4*>(a.x + r * a.pitch + 2 * (int64_t)col[i]);
        gs[i] = s[col[i] / 128];
        ps[i] = s[(a.inner + col[i]) / 128];
    }
#pragma unroll
    for (int i = 0; i < kSwigluUnits; ++i) {
        const bool in = row[i] >= 0;
        const int64_t r = max(row[i], 0);
        float gate[8], up[8], d[8];
        read_codes(g[i], gs[i], gate);
        read_codes(p[i], ps[i], up);
        unpack8<FP16>(dz[i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 s = sigmoid_and_rest(gate[j]);
            const float ds = d[j] * s.x, x = gate[j];
            gate[j] = ds * up[j] * fmaf(x, s.y, 1.0f);
            up[j] = ds * x;
        }
        uint8_t* out = a.d + r * 4 * a.inner;
        if constexpr (STRADDLE) {
            const bool second = at[i] >= a.inner;
#pragma unroll
            for (int j = 0; j < 8; ++j) gate[j] = second ? up[j] : gate[j];
            if (in) st_v4(out + 2 * (int64_t)at[i], pack8<FP16>(gate));
            write_codes(gate, block_top(gate), in, a.q + r * 2 * a.inner + at[i], a.scales + r * a.row_blocks + at[i] / 128);
        } else {
            if (in) {
                st_v4(out + 2 * (int64_t)col[i], pack8<FP16>(gate));
                st_v4(out + 2 * (int64_t)(a.inner + col[i]), pack8<FP16>(up));
            }
            if constexpr (QUANTISE) {
                uint8_t* q = a.q + r * 2 * a.inner;
                float* scales = a.scales + r * a.row_blocks;
                write_codes(gate, block_top(gate), in, q + col[i], scales + col[i] / 128);
                write_codes(up, block_top(up), in, q + a.inner + col[i], scales + (a.inner + col[i]) / 128);
            }
        }
    }
}

unsigned swiglu_grid(const SwigluArgs& a)
{
    const int64_t per_cta = kSwigluTeams * kSwigluUnits;
    return (unsigned)(((int64_t)a.rows * a.per_row + per_cta - 1) / per_cta);
}

// What forward and backward check alike; `x` names the 16-bit input, of `width` columns.
int check_swiglu(const char* who, const char* x, const SwigluArgs& a, int64_t rows, int64_t stride, int64_t width, int dtype,
                 const int32_t* end)
{
    if (dtype != EP_BF16 && dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "%s: dtype=%d is neither EP_BF16 nor EP_FP16", who, dtype);
    if (a.inner < 16 || a.inner % 16 != 0 || a.inner > 1 << 20)
        return layer_fail(EP_ERR_ARG, "%s: inner=%d is not a multiple of 16 in 16..2^20", who, a.inner);
    if (rows < 0 || rows >= (int64_t)1 << 31 || rows * (a.z_blocks + a.row_blocks) >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: rows=%lld of %d blocks reach 2^31", who, (long long)rows, a.z_blocks + a.row_blocks);
    if (end && !layer_aligned(end, 4)) return layer_fail(EP_ERR_ARG, "%s: rows_end is not 4-byte aligned", who);
    if (rows == 0) return EP_OK;
    if (!layer_aligned(a.x, 16) || stride < width || stride % 8 != 0)
        return layer_fail(EP_ERR_ARG, "%s: %s is NULL, not 16-byte aligned, or its row stride %lld is below %lld or not a "
                          "multiple of 8", who, x, (long long)stride, (long long)width);
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" int ep_swiglu_saved(const void* gate_up, int64_t stride, int dtype, int64_t rows, int inner,
                               const int32_t* rows_end, void* q, float* scales, void* saved, float* saved_scales,
                               void* stream)
{
    using namespace ep;
    const char* who = "ep_swiglu_saved";
    SwigluArgs a{};
    a.x = (const uint8_t*)gate_up; a.inner = inner; a.end = rows_end;
    a.z_blocks = (int)(((int64_t)inner + 127) / 128); a.row_blocks = (int)((2 * (int64_t)inner + 127) / 128);
    if (int rc = check_swiglu(who, "gate_up", a, rows, stride, 2 * (int64_t)inner, dtype, rows_end)) return rc;
    if (rows == 0) return EP_OK;
    if (!layer_aligned(q, 16) || !layer_aligned(saved, 16) || !layer_aligned(scales, 4) || !layer_aligned(saved_scales, 4))
        return layer_fail(EP_ERR_ARG, "%s: q, saved or a scale array is NULL or misaligned", who);
    a.q = (uint8_t*)q; a.scales = scales; a.saved = (uint8_t*)saved; a.saved_scales = saved_scales;
    a.pitch = 2 * stride; a.rows = (int)rows;
    const bool straddle = inner % 128 != 0, fp16 = dtype == EP_FP16;
    set_per_row(a, straddle ? a.z_blocks + a.row_blocks : a.z_blocks);
    const dim3 grid(swiglu_grid(a)), threads(kSwigluThreads);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (straddle)
        e = fp16 ? launch_dependent(ep_swiglu_saved_kernel<true, true>, grid, threads, 0, s, a)
                 : launch_dependent(ep_swiglu_saved_kernel<false, true>, grid, threads, 0, s, a);
    else
        e = fp16 ? launch_dependent(ep_swiglu_saved_kernel<true, false>, grid, threads, 0, s, a)
                 : launch_dependent(ep_swiglu_saved_kernel<false, false>, grid, threads, 0, s, a);
    return layer_cuda(e, "ep_swiglu_saved: launch");
}

extern "C" int ep_swiglu_saved_backward(const void* saved, const float* saved_scales, const void* dz, int64_t dz_stride,
                                        int dtype, int64_t rows, int inner, const int32_t* rows_end, void* d_gate_up,
                                        void* q, float* scales, void* stream)
{
    using namespace ep;
    const char* who = "ep_swiglu_saved_backward";
    SwigluArgs a{};
    a.x = (const uint8_t*)dz; a.inner = inner; a.end = rows_end;
    a.z_blocks = (int)(((int64_t)inner + 127) / 128); a.row_blocks = (int)((2 * (int64_t)inner + 127) / 128);
    if (int rc = check_swiglu(who, "dz", a, rows, dz_stride, inner, dtype, rows_end)) return rc;
    if (rows == 0) return EP_OK;
    if (!layer_aligned(saved, 16) || !layer_aligned(saved_scales, 4) || !layer_aligned(d_gate_up, 16))
        return layer_fail(EP_ERR_ARG, "%s: saved, saved_scales or d_gate_up is NULL or misaligned", who);
    if ((q != nullptr) != (scales != nullptr) || (q && (!layer_aligned(q, 16) || !layer_aligned(scales, 4))))
        return layer_fail(EP_ERR_ARG, "%s: q and scales are not both given and aligned, nor both NULL", who);
    a.saved_in = (const uint8_t*)saved; a.saved_in_scales = saved_scales;
    a.d = (uint8_t*)d_gate_up; a.q = (uint8_t*)q; a.scales = scales;
    a.pitch = 2 * dz_stride; a.rows = (int)rows;
    const bool straddle = q && inner % 128 != 0, fp16 = dtype == EP_FP16;
    set_per_row(a, straddle ? a.row_blocks : a.z_blocks);
    const dim3 grid(swiglu_grid(a)), threads(kSwigluThreads);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (straddle)
        e = fp16 ? launch_dependent(ep_swiglu_backward_kernel<true, true, true>, grid, threads, 0, s, a)
                 : launch_dependent(ep_swiglu_backward_kernel<false, true, true>, grid, threads, 0, s, a);
    else if (q)
        e = fp16 ? launch_dependent(ep_swiglu_backward_kernel<true, true, false>, grid, threads, 0, s, a)
                 : launch_dependent(ep_swiglu_backward_kernel<false, true, false>, grid, threads, 0, s, a);
    else
        e = fp16 ? launch_dependent(ep_swiglu_backward_kernel<true, false, false>, grid, threads, 0, s, a)
                 : launch_dependent(ep_swiglu_backward_kernel<false, false, false>, grid, threads, 0, s, a);
    return layer_cuda(e, "ep_swiglu_saved_backward: launch");
}
