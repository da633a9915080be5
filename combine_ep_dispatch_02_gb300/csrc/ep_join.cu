// ep_join.cu -- the norm after a block, joined through its gate to the scaled residual, with the norm before the
// next block; and the gradient of both.
//
//   u = y * rs(y) * post_weight          rs(v) = 1 / sqrt(mean(v^2) + eps); u = y without that norm
//   h = residual_scale * residual + gate * u
//   n = h * rs(h) * pre_weight           in 16 bits, or as e4m3 codes with one FP32 scale per 128 elements
//
//   D = dh + rs(h) * (g - x * mean(g * x))   with g = dn * pre_weight, x = h * rs(h)
//   dresidual = residual_scale * D;  dgate = D * u, summed to the gate's shape;  dpre = sum over rows of dn * x
//   dy = rs(y) * (p - v * mean(p * v))       with p = D * gate * post_weight, v = y * rs(y);  dpost = sum of D * gate * v
//
// All in FP32; each output is rounded once.  mean(p * v) is the mean of gate * D * u, so that a row's own gate and the
// norm share one sum.
#include "ep_layer.cuh"

namespace ep {
namespace {

struct JoinArgs {
    const uint8_t* y;
    const uint8_t* residual;
    const void* post_weight;    // NULL: no norm after the block
    const uint8_t* gate;        // NULL with EP_GATE_NONE
    const void* pre_weight;     // NULL: no norm before the next block
    const uint8_t* h_in;        // backward
    const uint8_t* dh;
    const uint8_t* dn;
    const float* post_rstd_in;
    const float* pre_rstd_in;
    uint8_t* h;
    uint8_t* n;
    uint8_t* q;
    float* scales;
    float* post_rstd;
    float* pre_rstd;
    uint8_t* dy;
    uint8_t* dresidual;
    uint8_t* dgate_element;
    float* dgate_row;
    float* partial;             // [CTAs][3][hidden]: sums for post_weight, gate, pre_weight
    int64_t rows, y_pitch, r_pitch, g_pitch, dh_pitch, dn_pitch;   // pitches in bytes
    int hidden, vecs, blocks;   // 16-byte vectors and 128-element blocks of a row
    int gate_kind, post_fp32, gate_fp32, pre_fp32;
    float residual_scale, eps;
};

constexpr int kJoinWarpsPerCta = 4;    // rows of a CTA when a row is one warp's
constexpr int kJoinMaxThreads = 512;
constexpr int kJoinMaxHidden = kJoinMaxThreads * 8 * 8;
constexpr int kJoinBackMaxThreads = 1024;
constexpr int kJoinBackMaxHidden = kJoinBackMaxThreads * 8;   // a vector of 8 columns per thread

// Eight values of a vector along the channels: FP32, or of the rows' type.
template <bool FP16>
__device__ __forceinline__ void load_channels(const void* p, int fp32, int v, float (&w)[8])
{
    if (fp32) {
        const float4* wp = reinterpret_cast<const float4*>(p) + 2 * v;
        const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
        w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
        w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
    } else {
        unpack8<FP16>(__ldg(reinterpret_cast<const uint4*>(p) + v), w);
    }
}

// Sum over a row's threads, a warp or a CTA; `part` holds 32 floats that no earlier sum of the row uses.
template <bool WARP>
__device__ __forceinline__ float row_sum(float sum, float* part)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    return sum;
}

// A row by one warp (WARP) or by the whole CTA; VPT vectors per thread.
template <bool FP16, bool WARP, int VPT>
__global__ void __launch_bounds__(WARP ? 32 * kJoinWarpsPerCta : kJoinMaxThreads) ep_join_kernel(const JoinArgs a)
{
    __shared__ float part[2][32];
    const int lane = threadIdx.x & 31;
    const int t = WARP ? lane : threadIdx.x;
    const int stride = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * kJoinWarpsPerCta + (threadIdx.x >> 5) : blockIdx.x;
    follow_predecessor();
    if (WARP && row >= a.rows) return;
    float f[VPT][8];
    uint4 res[VPT], el[VPT];
    {
        uint4 vy[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * stride + t;
            vy[i] = res[i] = el[i] = make_uint4(0, 0, 0, 0);
            if (v < a.vecs) {
                vy[i] = *reinterpret_cast<const uint4*>(a.y + row * a.y_pitch + 16 * (int64_t)v);
                res[i] = *reinterpret_cast<const uint4*>(a.residual + row * a.r_pitch + 16 * (int64_t)v);
                if (a.gate_kind == EP_GATE_ELEMENT)
                    el[i] = *reinterpret_cast<const uint4*>(a.gate + row * a.g_pitch + 16 * (int64_t)v);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) unpack8<FP16>(vy[i], f[i]);
    }
    float row_gate = a.gate_kind == EP_GATE_ROW ? reinterpret_cast<const float*>(a.gate)[row] : 1.0f;
    if (a.post_weight) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
        sum = row_sum<WARP>(sum, part[0]);
        const float rstd = __frsqrt_rn(__fdiv_rn(sum, (float)a.hidden) + a.eps);
        if (t == 0) a.post_rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * stride + t;
            float w[8] = {};
            if (v < a.vecs) load_channels<FP16>(a.post_weight, a.post_fp32, v, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * rstd * w[j];
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * stride + t;
        float r[8], g[8];
        unpack8<FP16>(res[i], r);
        if (a.gate_kind == EP_GATE_ELEMENT) {
            unpack8<FP16>(el[i], g);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = row_gate;
            if (a.gate_kind == EP_GATE_CHANNEL && v < a.vecs) load_channels<FP16>(a.gate, a.gate_fp32, v, g);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[i][j] = v < a.vecs ? fmaf(a.residual_scale, r[j], g[j] * f[i][j]) : 0.0f;
            sum = fmaf(f[i][j], f[i][j], sum);
        }
        if (v < a.vecs) *reinterpret_cast<uint4*>(a.h + (row * a.vecs + v) * 16) = pack8<FP16>(f[i]);
    }
    if (!a.pre_weight) return;
    sum = row_sum<WARP>(sum, part[1]);
    const float rstd = __frsqrt_rn(__fdiv_rn(sum, (float)a.hidden) + a.eps);
    if (t == 0) a.pre_rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * stride + t;
        const bool in = v < a.vecs;
        float w[8] = {};
        if (in) load_channels<FP16>(a.pre_weight, a.pre_fp32, v, w);
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[i][j] = f[i][j] * rstd * w[j];
            m = fmaxf(m, in ? fabsf(f[i][j]) : 0.0f);
        }
        if (in && a.n) *reinterpret_cast<uint4*>(a.n + (row * a.vecs + v) * 16) = pack8<FP16>(f[i]);
        if (!a.q) continue;
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float scale = e4m3_block_scale(m);
        const float inv = __frcp_rn(scale);
        if (in) {
            const uint2 q = make_uint2(e4m3x4_scaled(f[i][0], f[i][1], f[i][2], f[i][3], scale, inv),
                                       e4m3x4_scaled(f[i][4], f[i][5], f[i][6], f[i][7], scale, inv));
            *reinterpret_cast<uint2*>(a.q + (row * a.vecs + v) * 8) = q;
            if ((v & 15) == 0) a.scales[row * a.blocks + (v >> 4)] = scale;
        }
    }
}

// 16 bytes of global memory into shared memory, asynchronously; a thread's copies are grouped by copies_commit() and
// copies_wait<N>() returns when all but the newest N groups have arrived, for the thread that made them.
__device__ __forceinline__ void copy16(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// Rows blockIdx.x, + gridDim.x, ... by one CTA, a vector of 8 columns per thread: the sums over rows stay in registers
// and leave once per CTA.  Rows are on their way through STAGES stages of shared memory, of which a thread fills and
// reads its own vectors only, so that no barrier passes between copy and use; registers hold the three sums and one
// gradient, and what a later pass over the row needs is read from the stage again.
enum { kSlotH, kSlotDn, kSlotDh, kSlotY, kSlotGate };   // a stage's vectors of a thread; the last for a gate per element

template <bool FP16, bool WARP, int STAGES>
__global__ void __launch_bounds__(WARP ? 32 : kJoinBackMaxThreads) ep_join_backward_kernel(const JoinArgs a)
{
    extern __shared__ uint4 staged[];
    __shared__ float part[4][32];
    const int t = threadIdx.x;
    const bool in = t < a.vecs;
    const int64_t at = 16 * (int64_t)t;
    const int slots = a.gate_kind == EP_GATE_ELEMENT ? 5 : 4;
    const float inv_hidden = __frcp_rn((float)a.hidden);
    follow_predecessor();
    auto fetch = [&](int64_t row, int stage) {
        if (in && row < a.rows) {
            uint4* to = staged + stage * slots * blockDim.x + t;
            if (a.pre_weight) {
                copy16(to + kSlotH * blockDim.x, a.h_in + row * 16 * a.vecs + at);
                copy16(to + kSlotDn * blockDim.x, a.dn + row * a.dn_pitch + at);
            }
            if (a.dh) copy16(to + kSlotDh * blockDim.x, a.dh + row * a.dh_pitch + at);
            copy16(to + kSlotY * blockDim.x, a.y + row * a.y_pitch + at);
            if (a.gate_kind == EP_GATE_ELEMENT) copy16(to + kSlotGate * blockDim.x, a.gate + row * a.g_pitch + at);
        }
        copies_commit();
    };
    float dpost[8] = {}, dgate[8] = {}, dpre[8] = {};
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
    int parity = 0, stage = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 2) {
        const float pre = a.pre_weight ? a.pre_rstd_in[row] : 0.0f;
        const float post = a.post_weight ? a.post_rstd_in[row] : 1.0f;
        const float row_gate = a.gate_kind == EP_GATE_ROW ? reinterpret_cast<const float*>(a.gate)[row] : 1.0f;
        const uint4* mine = staged + stage * slots * blockDim.x + t;
        copies_wait<STAGES - 1>();
        float mean = 0.0f;
        if (a.pre_weight) {
            float sum = 0.0f;
            if (in) {
                float x[8], g[8], w[8];
                unpack8<FP16>(mine[kSlotH * blockDim.x], x);
                unpack8<FP16>(mine[kSlotDn * blockDim.x], g);
                load_channels<FP16>(a.pre_weight, a.pre_fp32, t, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float gx = g[j] * (x[j] * pre);
                    dpre[j] += gx;
                    sum = fmaf(gx, w[j], sum);
                }
            }
            mean = row_sum<WARP>(sum, part[parity]) * inv_hidden;
        }
        float d[8], sum = 0.0f;
        if (in) {
            if (a.dh) {
                unpack8<FP16>(mine[kSlotDh * blockDim.x], d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = 0.0f;
            }
            if (a.pre_weight) {
                float x[8], g[8], w[8];
                unpack8<FP16>(mine[kSlotH * blockDim.x], x);
                unpack8<FP16>(mine[kSlotDn * blockDim.x], g);
                load_channels<FP16>(a.pre_weight, a.pre_fp32, t, w);
                const float along = -mean * pre;
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaf(pre, fmaf(x[j], along, g[j] * w[j]), d[j]);
            }
            if (a.dresidual) {
                float r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = a.residual_scale * d[j];
                st_v4(a.dresidual + row * 16 * a.vecs + at, pack8<FP16>(r));
            }
            float v[8], u[8];
            unpack8<FP16>(mine[kSlotY * blockDim.x], v);
            if (a.post_weight) {
                load_channels<FP16>(a.post_weight, a.post_fp32, t, u);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = 1.0f;
            }
            // u: the gradient for the gate; d: that for y's norm, times the gate
            float gate[8];
            if (a.gate_kind == EP_GATE_ELEMENT) {
                unpack8<FP16>(mine[kSlotGate * blockDim.x], gate);
            } else if (a.gate_kind == EP_GATE_CHANNEL) {
                load_channels<FP16>(a.gate, a.gate_fp32, t, gate);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) gate[j] = row_gate;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] *= post;
                const float w = u[j], p = d[j] * gate[j];
                u[j] = d[j] * (v[j] * w);
                dgate[j] += u[j];
                dpost[j] = fmaf(p, v[j], dpost[j]);
                d[j] = p * w;
                sum = a.gate_kind == EP_GATE_ROW ? sum + u[j] : fmaf(d[j], v[j], sum);
            }
            if (a.gate_kind == EP_GATE_ELEMENT) st_v4(a.dgate_element + row * 16 * a.vecs + at, pack8<FP16>(u));
        }
        mean = 0.0f;
        if (a.post_weight || a.gate_kind == EP_GATE_ROW) {
            sum = row_sum<WARP>(sum, part[parity + 1]);
            if (a.gate_kind == EP_GATE_ROW) {
                if (t == 0) a.dgate_row[row] = sum;
                sum *= row_gate;
            }
            mean = sum * inv_hidden;
        }
        if (in) {
            if (a.post_weight) {
                float v[8];
                unpack8<FP16>(mine[kSlotY * blockDim.x], v);
                const float along = -mean * post;
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = post * fmaf(v[j], along, d[j]);
            }
            st_v4(a.dy + row * 16 * a.vecs + at, pack8<FP16>(d));
        }
        fetch(row + (int64_t)STAGES * gridDim.x, stage);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    if (!in) return;
    float* out = a.partial + (int64_t)blockIdx.x * 3 * a.hidden + 8 * t;
    auto leave = [&](const float (&s)[8], int which) {
        float4* p = reinterpret_cast<float4*>(out + (int64_t)which * a.hidden);
        p[0] = make_float4(s[0], s[1], s[2], s[3]);
        p[1] = make_float4(s[4], s[5], s[6], s[7]);
    };
    if (a.post_weight) leave(dpost, 0);
    if (a.gate_kind == EP_GATE_CHANNEL) leave(dgate, 1);
    if (a.pre_weight) leave(dpre, 2);
}

// The CTAs' sums, added in their order: thread (column, part) adds a part of the CTAs, and the parts are added in
// order.  blockIdx.y is the sum.
struct JoinSumArgs {
    const float* partial;
    float* out[3];
    int ctas, hidden;
};

constexpr int kSumColumns = 32, kSumParts = 16;

__global__ void __launch_bounds__(kSumColumns * kSumParts) ep_join_sum_kernel(const JoinSumArgs a)
{
    __shared__ float part[kSumParts][kSumColumns];
    const int c = blockIdx.x * kSumColumns + threadIdx.x;
    follow_predecessor();
    float* out = a.out[blockIdx.y];
    if (!out) return;
    const int lo = a.ctas * (int)threadIdx.y / kSumParts, hi = a.ctas * ((int)threadIdx.y + 1) / kSumParts;
    float s = 0.0f;
    if (c < a.hidden) {
        const float* p = a.partial + (int64_t)blockIdx.y * a.hidden + c;
#pragma unroll 8
        for (int i = lo; i < hi; ++i) s += p[(int64_t)i * 3 * a.hidden];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || c >= a.hidden) return;
#pragma unroll
    for (int i = 1; i < kSumParts; ++i) s += part[i][threadIdx.x];
    out[c] = s;
}

template <bool FP16, bool WARP>
cudaError_t launch_join(const JoinArgs& a, int vpt, int threads, cudaStream_t s)
{
    const unsigned grid = (unsigned)(WARP ? (a.rows + kJoinWarpsPerCta - 1) / kJoinWarpsPerCta : a.rows);
    const dim3 block(threads);
    if constexpr (WARP) {
        if (vpt == 1) return launch_dependent(ep_join_kernel<FP16, true, 1>, dim3(grid), block, 0, s, a);
        if (vpt == 2) return launch_dependent(ep_join_kernel<FP16, true, 2>, dim3(grid), block, 0, s, a);
        return launch_dependent(ep_join_kernel<FP16, true, 4>, dim3(grid), block, 0, s, a);
    } else {
        if (vpt == 4) return launch_dependent(ep_join_kernel<FP16, false, 4>, dim3(grid), block, 0, s, a);
        return launch_dependent(ep_join_kernel<FP16, false, 8>, dim3(grid), block, 0, s, a);
    }
}

// CTAs of the gradient's kernel: as many as the SMs hold at once, but no fewer than kRowsPerCta rows to each, because
// every CTA leaves three rows of sums.
constexpr int kRowsPerCta = 4;

int join_backward_ctas(int64_t rows, int hidden, int sms)
{
    const int threads = (hidden / 8 + 31) / 32 * 32;
    const int64_t fit = (int64_t)sms * (threads > 512 ? 1 : threads > 256 ? 2 : threads > 128 ? 4 : 8);
    const int64_t want = (rows + kRowsPerCta - 1) / kRowsPerCta;
    const int64_t least = rows < sms ? rows : sms;
    return (int)(want < least ? least : want < fit ? want : fit);
}

template <bool FP16, bool WARP, int STAGES>
cudaError_t launch_join_backward(const JoinArgs& a, int ctas, int threads, cudaStream_t s)
{
    const cudaError_t e = allow_all_shared<ep_join_backward_kernel<FP16, WARP, STAGES>>();
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)STAGES * (a.gate_kind == EP_GATE_ELEMENT ? 5 : 4) * threads * 16;
    return launch_dependent(ep_join_backward_kernel<FP16, WARP, STAGES>, dim3(ctas), dim3(threads), smem, s, a);
}

template <bool FP16>
cudaError_t launch_join_backward(const JoinArgs& a, int ctas, cudaStream_t s)
{
    const int threads = (a.vecs + 31) / 32 * 32;
    if (threads == 32) return launch_join_backward<FP16, true, 3>(a, ctas, threads, s);
    // a third stage of five vectors to a thread would pass a CTA's shared memory
    if (threads > 896) return launch_join_backward<FP16, false, 2>(a, ctas, threads, s);
    return launch_join_backward<FP16, false, 3>(a, ctas, threads, s);
}

bool row_ok(const void* p, int64_t stride, int hidden)
{
    return layer_aligned(p, 16) && stride >= hidden && stride % 8 == 0;
}

// What forward and backward check alike, and the arguments that they share.
int check_join(const char* who, const ep_join* j, int max_hidden, JoinArgs& a)
{
    if (!j) return layer_fail(EP_ERR_ARG, "%s: join is NULL", who);
    if (j->dtype != EP_BF16 && j->dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "%s: dtype=%d is neither EP_BF16 nor EP_FP16", who, j->dtype);
    if (j->hidden < 16 || j->hidden > max_hidden || j->hidden % 16 != 0)
        return layer_fail(EP_ERR_ARG, "%s: hidden=%d is not a multiple of 16 in 16..%d", who, j->hidden, max_hidden);
    if (j->rows < 0 || j->rows >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: rows=%lld outside 0..2^31-1", who, (long long)j->rows);
    if (!(j->eps >= 0.0f)) return layer_fail(EP_ERR_ARG, "%s: eps=%g is negative or NaN", who, (double)j->eps);
    if (j->gate_kind < EP_GATE_NONE || j->gate_kind > EP_GATE_ELEMENT)
        return layer_fail(EP_ERR_ARG, "%s: gate_kind=%d is none of EP_GATE_*", who, j->gate_kind);
    if ((j->post_weight && !layer_aligned(j->post_weight, 16)) || (j->pre_weight && !layer_aligned(j->pre_weight, 16)))
        return layer_fail(EP_ERR_ARG, "%s: a weight is not 16-byte aligned", who);
    if (j->rows > 0) {
        if (!row_ok(j->y, j->y_stride, j->hidden))
            return layer_fail(EP_ERR_ARG, "%s: y is NULL, not 16-byte aligned, or its row stride %lld is below hidden or not "
                              "a multiple of 8", who, (long long)j->y_stride);
        if (j->gate_kind == EP_GATE_ROW ? !layer_aligned(j->gate, 4)
            : j->gate_kind == EP_GATE_CHANNEL ? !layer_aligned(j->gate, 16)
            : j->gate_kind == EP_GATE_ELEMENT && !row_ok(j->gate, j->gate_stride, j->hidden))
            return layer_fail(EP_ERR_ARG, "%s: gate is NULL, misaligned, or its row stride %lld is below hidden or not a "
                              "multiple of 8", who, (long long)j->gate_stride);
    }
    a.y = (const uint8_t*)j->y; a.gate = (const uint8_t*)j->gate;
    a.post_weight = j->post_weight; a.pre_weight = j->pre_weight;
    a.rows = j->rows; a.y_pitch = 2 * j->y_stride; a.g_pitch = 2 * j->gate_stride;
    a.hidden = j->hidden; a.vecs = j->hidden / 8; a.blocks = (j->hidden + 127) / 128;
    a.gate_kind = j->gate_kind; a.post_fp32 = j->post_fp32; a.gate_fp32 = j->gate_fp32; a.pre_fp32 = j->pre_fp32;
    a.residual_scale = j->residual_scale; a.eps = j->eps;
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" int ep_rms_norm_join(const ep_join* join, const void* residual, int64_t residual_stride, void* h, void* n,
                                void* q, float* scales, float* post_rstd, float* pre_rstd, void* stream)
{
    using namespace ep;
    const char* who = "ep_rms_norm_join";
    JoinArgs a{};
    if (int rc = check_join(who, join, kJoinMaxHidden, a)) return rc;
    if (a.rows == 0) return EP_OK;
    if (!row_ok(residual, residual_stride, a.hidden))
        return layer_fail(EP_ERR_ARG, "%s: residual is NULL, not 16-byte aligned, or its row stride %lld is below hidden or "
                          "not a multiple of 8", who, (long long)residual_stride);
    if (!layer_aligned(h, 16) || (n && !layer_aligned(n, 16)))
        return layer_fail(EP_ERR_ARG, "%s: h is NULL, or h or n is not 16-byte aligned", who);
    if ((q != nullptr) != (scales != nullptr) || (q && (!layer_aligned(q, 16) || !layer_aligned(scales, 4))))
        return layer_fail(EP_ERR_ARG, "%s: q and scales are not both given and aligned, nor both NULL", who);
    if (!a.pre_weight && (n || q)) return layer_fail(EP_ERR_ARG, "%s: n or q is wanted without pre_weight", who);
    if ((a.post_weight && !layer_aligned(post_rstd, 4)) || (a.pre_weight && !layer_aligned(pre_rstd, 4)))
        return layer_fail(EP_ERR_ARG, "%s: post_rstd or pre_rstd is NULL or misaligned", who);
    a.residual = (const uint8_t*)residual; a.r_pitch = 2 * residual_stride;
    a.h = (uint8_t*)h; a.n = (uint8_t*)n; a.q = (uint8_t*)q; a.scales = scales;
    a.post_rstd = post_rstd; a.pre_rstd = pre_rstd;
    const bool fp16 = join->dtype == EP_FP16;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (a.vecs <= 128) {   // a row per warp
        const int vpt = a.vecs <= 32 ? 1 : a.vecs <= 64 ? 2 : 4;
        e = fp16 ? launch_join<true, true>(a, vpt, 32 * kJoinWarpsPerCta, s)
                 : launch_join<false, true>(a, vpt, 32 * kJoinWarpsPerCta, s);
    } else {
        const int vpt = a.vecs <= 4 * kJoinMaxThreads ? 4 : 8;
        const int threads = ((a.vecs + vpt - 1) / vpt + 31) / 32 * 32;
        e = fp16 ? launch_join<true, false>(a, vpt, threads, s) : launch_join<false, false>(a, vpt, threads, s);
    }
    return layer_cuda(e, "ep_rms_norm_join: launch");
}

extern "C" size_t ep_rms_norm_join_workspace_bytes(int64_t rows, int hidden)
{
    using namespace ep;
    if (rows <= 0 || rows >= (int64_t)1 << 31 || hidden < 16 || hidden > kJoinBackMaxHidden || hidden % 16 != 0) return 0;
    return (size_t)join_backward_ctas(rows, hidden, layer_num_sms()) * 3 * hidden * sizeof(float);
}

extern "C" int ep_rms_norm_join_backward(const ep_join* join, const void* h, const float* post_rstd, const float* pre_rstd,
                                         const void* dh, int64_t dh_stride, const void* dn, int64_t dn_stride, void* dy,
                                         void* dresidual, float* dpost_weight, void* dgate, float* dpre_weight,
                                         void* workspace, size_t workspace_bytes, void* stream)
{
    using namespace ep;
    const char* who = "ep_rms_norm_join_backward";
    JoinArgs a{};
    if (int rc = check_join(who, join, kJoinBackMaxHidden, a)) return rc;
    if ((dn != nullptr) != (a.pre_weight != nullptr) && a.rows > 0)
        return layer_fail(EP_ERR_ARG, "%s: dn and pre_weight are not both given, nor both NULL", who);
    if (!dh && !dn && a.rows > 0) return layer_fail(EP_ERR_ARG, "%s: neither dh nor dn is given", who);
    if ((a.post_weight && !layer_aligned(dpost_weight, 4)) || (a.pre_weight && !layer_aligned(dpre_weight, 4)) ||
        (a.gate_kind == EP_GATE_CHANNEL && !layer_aligned(dgate, 4)))
        return layer_fail(EP_ERR_ARG, "%s: the gradient of a weight or of the channels' gate is NULL or misaligned", who);
    const bool fp16 = join->dtype == EP_FP16;
    cudaStream_t s = (cudaStream_t)stream;
    JoinSumArgs sums{(const float*)workspace,
                     {a.post_weight ? dpost_weight : nullptr, a.gate_kind == EP_GATE_CHANNEL ? (float*)dgate : nullptr,
                      a.pre_weight ? dpre_weight : nullptr}, 0, a.hidden};
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) {
        if ((dh && !row_ok(dh, dh_stride, a.hidden)) || (dn && !row_ok(dn, dn_stride, a.hidden)))
            return layer_fail(EP_ERR_ARG, "%s: dh or dn is not 16-byte aligned, or its row stride is below hidden or not a "
                              "multiple of 8", who);
        if ((dn && !layer_aligned(h, 16)) || !layer_aligned(dy, 16) || (dresidual && !layer_aligned(dresidual, 16)))
            return layer_fail(EP_ERR_ARG, "%s: h, dy or dresidual is NULL or misaligned", who);
        if ((a.gate_kind == EP_GATE_ELEMENT && !layer_aligned(dgate, 16)) || (a.gate_kind == EP_GATE_ROW && !layer_aligned(dgate, 4)))
            return layer_fail(EP_ERR_ARG, "%s: dgate is NULL or misaligned", who);
        if ((a.post_weight && !layer_aligned(post_rstd, 4)) || (a.pre_weight && !layer_aligned(pre_rstd, 4)))
            return layer_fail(EP_ERR_ARG, "%s: post_rstd or pre_rstd is NULL or misaligned", who);
        const int sms = layer_num_sms();
        if (sms == 0) return layer_fail(EP_ERR_CUDA, "%s: cannot tell the current device's multiprocessors", who);
        sums.ctas = join_backward_ctas(a.rows, a.hidden, sms);
        const size_t need = (size_t)sums.ctas * 3 * a.hidden * sizeof(float);
        if (!layer_aligned(workspace, 16) || workspace_bytes < need)
            return layer_fail(EP_ERR_ARG, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", who, workspace_bytes, need);
        a.h_in = (const uint8_t*)h; a.dh = (const uint8_t*)dh; a.dn = (const uint8_t*)dn;
        a.dh_pitch = 2 * dh_stride; a.dn_pitch = 2 * dn_stride;
        a.post_rstd_in = post_rstd; a.pre_rstd_in = pre_rstd;
        a.dy = (uint8_t*)dy; a.dresidual = (uint8_t*)dresidual;
        if (a.gate_kind == EP_GATE_ELEMENT) a.dgate_element = (uint8_t*)dgate;
        if (a.gate_kind == EP_GATE_ROW) a.dgate_row = (float*)dgate;
        a.partial = (float*)workspace;
        e = fp16 ? launch_join_backward<true>(a, sums.ctas, s) : launch_join_backward<false>(a, sums.ctas, s);
    }
    if (e == cudaSuccess && (sums.out[0] || sums.out[1] || sums.out[2]))
        e = launch_dependent(ep_join_sum_kernel, dim3((a.hidden + kSumColumns - 1) / kSumColumns, 3),
                             dim3(kSumColumns, kSumParts), 0, s, sums);
    return layer_cuda(e, "ep_rms_norm_join_backward: launch");
}
