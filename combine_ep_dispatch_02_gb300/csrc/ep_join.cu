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
//
// Measured: 32768 rows of 7168, codes out, 289 us (5.7 TB/s): bytes take 244 us, and three quarters of the issue slots
// are taken.  One row 3.4 us.  The gradient of 8192 rows of 7168 143 us (4.9 TB/s; bytes 104): the CTA's 16 warps, all
// that its 126 registers and 200 KB of rows on their way allow, wait for one another at a sum and for their stages, and
// 9 us go to the sums over CTAs.
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

constexpr int kJoinMaxThreads = 512;   // of a wide row's CTA
constexpr int kJoinMaxHidden = kJoinMaxThreads * 8 * 8;

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

// Two sums over a row's threads, a warp or a CTA of up to 16; `part` holds 16 pairs that no thread still reads.  Half of a
// warp adds up one of them, the other half the other.
template <bool WARP>
__device__ __forceinline__ float2 row_sums(float2 s, float* part)
{
    const int lane = threadIdx.x & 31;
    const bool upper = lane & 16;
    float v = upper ? s.y : s.x;
    v += __shfl_xor_sync(0xffffffffu, upper ? s.x : s.y, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (!WARP) {
        if ((lane & 15) == 0) part[(lane & 16) + (threadIdx.x >> 5)] = v;
        __syncthreads();
        v = (lane & 15) < (int)(blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    const float other = __shfl_xor_sync(0xffffffffu, v, 16);
    return upper ? make_float2(other, v) : make_float2(v, other);
}

// 1 / sqrt(v): the approximation, off by two units, and one step of Newton's method.
__device__ __forceinline__ float root_of(float v)
{
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    const float e = fmaf(-v * r, r, 1.0f);   // not a number where v is 0 or infinite, whose roots are exact
    return fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
}

// ---- rows up to kJoinTeamHidden: one CTA of VPT vectors of 8 columns per thread walks rows blockIdx.x, + gridDim.x, ...
//
// Rows are on their way through STAGES stages of shared memory, of which a thread fills and reads its own vectors only,
// so that no barrier passes between copy and use.  The vectors along the channels (both weights and the channels' gate)
// lie there too.  A row needs two sums over its threads, the second from the first's result, and a CTA's sum costs
// some 400 cycles of shuffles and barrier; so the first sum of the next row is made together with the second of this one,
// and a row meets one barrier.  What bounds it is the instructions as much as the bytes: two vectors per thread halve what
// sums, roots and addresses cost an element, and FP32 arithmetic is done in pairs.

constexpr int kJoinTeamThreads = 512;
constexpr int kJoinTeamHidden = 16 * kJoinTeamThreads;

// A thread's vectors along the channels in shared memory: post_weight, gate, pre_weight, 16 bytes each or 32 for FP32.
struct Channels {
    uint4 *post, *gate, *pre;
};

__host__ __device__ inline int channel_vectors(const JoinArgs& a)   // 16-byte vectors of all three, per vector of a row
{
    return (a.post_weight ? 1 + (a.post_fp32 != 0) : 0) + (a.gate_kind == EP_GATE_CHANNEL ? 1 + (a.gate_fp32 != 0) : 0) +
           (a.pre_weight ? 1 + (a.pre_fp32 != 0) : 0);
}

template <int VPT>
__device__ __forceinline__ Channels fetch_channels(const JoinArgs& a, uint4* to)   // part of the first group of copies
{
    const int t = threadIdx.x, width = VPT * blockDim.x;
    auto fetch = [&](const void* from, int fp32) {
        uint4* at = to;
        to += width << (fp32 != 0);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * blockDim.x + t;
            if (v >= a.vecs) continue;
            if (fp32) {   // the second half of a vector's eight lies a row of vectors further on
                copy16(at + v, (const uint8_t*)from + 32 * v);
                copy16(at + width + v, (const uint8_t*)from + 32 * v + 16);
            } else {
                copy16(at + v, (const uint8_t*)from + 16 * v);
            }
        }
        return at + t;
    };
    Channels c{};
    if (a.post_weight) c.post = fetch(a.post_weight, a.post_fp32);
    if (a.gate_kind == EP_GATE_CHANNEL) c.gate = fetch(a.gate, a.gate_fp32);
    if (a.pre_weight) c.pre = fetch(a.pre_weight, a.pre_fp32);
    return c;
}

template <bool FP16, int VPT>
__device__ __forceinline__ void read_channels(const uint4* p, int fp32, int i, float2 (&w)[4])   // the thread's vector i
{
    p += i * blockDim.x;
    if (fp32) {
        const float4 lo = *reinterpret_cast<const float4*>(p), hi = *reinterpret_cast<const float4*>(p + VPT * blockDim.x);
        w[0] = make_float2(lo.x, lo.y);
        w[1] = make_float2(lo.z, lo.w);
        w[2] = make_float2(hi.x, hi.y);
        w[3] = make_float2(hi.z, hi.w);
    } else {
        unpack4x2<FP16>(*p, w);
    }
}

template <bool FP16, bool WARP, int VPT, int STAGES>
__global__ void __launch_bounds__(WARP ? 32 : kJoinTeamThreads, WARP ? 24 : 2) ep_join_team_kernel(const JoinArgs a)
{
    extern __shared__ uint4 staged[];
    __shared__ float part[2][32];
    const int t = threadIdx.x, threads = blockDim.x;
    const bool all = (VPT - 1) * threads + t < a.vecs;   // the thread's last vector exists; with two, the first always does
    const int64_t at = 16 * (int64_t)t, pitch = 16 * (int64_t)a.vecs, next_vector = 16 * (int64_t)threads;
    const bool element = a.gate_kind == EP_GATE_ELEMENT;
    const int slots = element ? 3 : 2, slot = VPT * threads;   // y, residual, the elements' gate
    const float inv_hidden = __frcp_rn((float)a.hidden);
    follow_predecessor();
    const Channels ch = fetch_channels<VPT>(a, staged + STAGES * slots * slot);
    uint4* const mine = staged + t;
    int64_t ahead = blockIdx.x;   // the next row to fetch
    const uint8_t *yp = a.y + ahead * a.y_pitch + at, *rp = a.residual + ahead * a.r_pitch + at;
    const uint8_t* gp = a.gate + (element ? ahead * a.g_pitch + at : 0);
    auto fetch = [&](int stage) {
        if (ahead < a.rows) {
            uint4* to = mine + stage * slots * slot;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (i + 1 == VPT && !all) break;
                copy16(to + i * threads, yp + i * next_vector);
                copy16(to + slot + i * threads, rp + i * next_vector);
                if (element) copy16(to + 2 * slot + i * threads, gp + i * next_vector);
            }
            ahead += gridDim.x;
            yp += gridDim.x * a.y_pitch;
            rp += gridDim.x * a.r_pitch;
            if (element) gp += gridDim.x * a.g_pitch;
        }
        copies_commit();
    };
    auto squares = [&](int stage) {   // of a row's y
        float2 s = both(0.0f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i + 1 == VPT && !all) break;
            float2 y[4];
            unpack4x2<FP16>(mine[stage * slots * slot + i * threads], y);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = fused2(y[j], y[j], s);
        }
        return s.x + s.y;
    };
    auto gate_of = [&](int64_t row) {
        return a.gate_kind == EP_GATE_ROW && row < a.rows ? reinterpret_cast<const float*>(a.gate)[row] : 1.0f;
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(i);
    float row_gate = gate_of(blockIdx.x), post = 1.0f;
    copies_wait<STAGES - 1>();
    if (a.post_weight) {
        post = root_of(fmaf(row_sums<WARP>(make_float2(squares(0), 0.0f), part[1]).x, inv_hidden, a.eps));
        if (t == 0) a.post_rstd[blockIdx.x] = post;
    }
    int parity = 0, stage = 0;
    int64_t out = blockIdx.x * pitch + at;   // bytes into h and n
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1, out += gridDim.x * pitch) {
        const float next_gate = gate_of(row + gridDim.x);
        float2 h[VPT][4], s = both(0.0f), sums = both(0.0f);
        const float2 scale = both(row_gate * post), along = both(a.residual_scale);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i + 1 == VPT && !all) {
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] = both(0.0f);
                break;
            }
            const uint4* from = mine + stage * slots * slot + i * threads;
            float2 r[4], w[4];
            unpack4x2<FP16>(from[0], h[i]);
            unpack4x2<FP16>(from[slot], r);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] = mul2(h[i][j], scale);
            if (a.post_weight) {
                read_channels<FP16, VPT>(ch.post, a.post_fp32, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] = mul2(h[i][j], w[j]);
            }
            if (element || a.gate_kind == EP_GATE_CHANNEL) {
                if (element) unpack4x2<FP16>(from[2 * slot], w);
                else read_channels<FP16, VPT>(ch.gate, a.gate_fp32, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[i][j] = mul2(h[i][j], w[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[i][j] = fused2(along, r[j], h[i][j]);
                s = fused2(h[i][j], h[i][j], s);
            }
            st_v4(a.h + out + i * next_vector, pack4x2<FP16>(h[i]));
        }
        sums.y = s.x + s.y;
        const int after = stage + 1 == STAGES ? 0 : stage + 1;
        copies_wait<STAGES - 2>();
        const bool another = row + gridDim.x < a.rows;
        if (a.post_weight && another) sums.x = squares(after);
        fetch(stage);
        stage = after;
        if (a.post_weight || a.pre_weight) sums = row_sums<WARP>(sums, part[parity]);
        if (a.post_weight) {
            post = root_of(fmaf(sums.x, inv_hidden, a.eps));
            if (t == 0 && another) a.post_rstd[row + gridDim.x] = post;
        }
        row_gate = next_gate;
        if (!a.pre_weight) continue;
        const float pre = root_of(fmaf(sums.y, inv_hidden, a.eps));
        if (t == 0) a.pre_rstd[row] = pre;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const bool in = i + 1 < VPT || all;
            float m = 0.0f;
            if (in) {
                float2 w[4];
                read_channels<FP16, VPT>(ch.pre, a.pre_fp32, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[i][j] = mul2(mul2(h[i][j], both(pre)), w[j]);
                    m = fmaxf(m, fmaxf(fabsf(h[i][j].x), fabsf(h[i][j].y)));
                }
                if (a.n) st_v4(a.n + out + i * next_vector, pack4x2<FP16>(h[i]));
            }
            if (!a.q) continue;
#pragma unroll
            for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float block = quick_block_scale(m), inv = quick_reciprocal(block);
            if (in) {
                const int v = i * threads + t;
                *reinterpret_cast<uint2*>(a.q + ((out - at) >> 1) + 8 * v) =
                    make_uint2(e4m3x4_near(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y, block, inv),
                               e4m3x4_near(h[i][2].x, h[i][2].y, h[i][3].x, h[i][3].y, block, inv));
                if ((t & 15) == 0) a.scales[row * a.blocks + (v >> 4)] = block;
            }
        }
    }
}

// The gradient.  The vectors along the channels lie in shared memory as FP32: pre_weight, and post_weight times the
// channels' gate.  One sum over rows, of q = D * v, gives both post_weight's gradient and the channels' gate's, each times
// the other; a row's own gate is a factor of all that follows D, and its gradient is the sum that the norm needs.  What a
// later pass over the row needs is read from its stage again.
enum { kSlotH, kSlotDn, kSlotDh, kSlotY, kSlotGate };   // a stage's vectors of a thread; the last for a gate per element
constexpr int kBackChannels = 4;                        // 16-byte vectors of both channel vectors, per vector of a row

template <bool FP16, bool WARP, int VPT, int STAGES>
__global__ void __launch_bounds__(WARP ? 32 : kJoinTeamThreads, 1) ep_join_backward_kernel(const JoinArgs a)
{
    extern __shared__ uint4 staged[];
    __shared__ float part[2][32];
    const int t = threadIdx.x, threads = blockDim.x;
    const bool all = (VPT - 1) * threads + t < a.vecs;   // as above
    const int64_t at = 16 * (int64_t)t, pitch = 16 * (int64_t)a.vecs, next_vector = 16 * (int64_t)threads;
    const bool element = a.gate_kind == EP_GATE_ELEMENT;
    const int slots = element ? 5 : 4, slot = VPT * threads;
    const float inv_hidden = __frcp_rn((float)a.hidden);
    follow_predecessor();
    uint4* const mine = staged + t;
    int64_t ahead = blockIdx.x;   // the next row to fetch
    const uint8_t *hp = a.h_in + ahead * pitch + at, *np = a.dn + ahead * a.dn_pitch + at, *dp = a.dh + ahead * a.dh_pitch + at,
                  *yp = a.y + ahead * a.y_pitch + at, *gp = a.gate + (element ? ahead * a.g_pitch + at : 0);
    auto fetch = [&](int stage) {
        if (ahead < a.rows) {
            uint4* to = mine + stage * slots * slot;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (i + 1 == VPT && !all) break;
                if (a.pre_weight) {
                    copy16(to + kSlotH * slot + i * threads, hp + i * next_vector);
                    copy16(to + kSlotDn * slot + i * threads, np + i * next_vector);
                }
                if (a.dh) copy16(to + kSlotDh * slot + i * threads, dp + i * next_vector);
                copy16(to + kSlotY * slot + i * threads, yp + i * next_vector);
                if (element) copy16(to + kSlotGate * slot + i * threads, gp + i * next_vector);
            }
            ahead += gridDim.x;
            hp += gridDim.x * pitch;
            np += gridDim.x * a.dn_pitch;
            dp += gridDim.x * a.dh_pitch;
            yp += gridDim.x * a.y_pitch;
            if (element) gp += gridDim.x * a.g_pitch;
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) fetch(i);
    float4* const channels = reinterpret_cast<float4*>(mine + STAGES * slots * slot);   // pre, then post * gate; two halves each
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (i + 1 == VPT && !all) break;
        const int v = i * threads + t;
        float pre[8], post[8], gate[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) pre[j] = post[j] = gate[j] = 1.0f;
        if (a.pre_weight) load_channels<FP16>(a.pre_weight, a.pre_fp32, v, pre);
        if (a.post_weight) load_channels<FP16>(a.post_weight, a.post_fp32, v, post);
        if (a.gate_kind == EP_GATE_CHANNEL) load_channels<FP16>(a.gate, a.gate_fp32, v, gate);
        float4* to = channels + i * threads;
        to[0] = make_float4(pre[0], pre[1], pre[2], pre[3]);
        to[slot] = make_float4(pre[4], pre[5], pre[6], pre[7]);
        to[2 * slot] = make_float4(post[0] * gate[0], post[1] * gate[1], post[2] * gate[2], post[3] * gate[3]);
        to[3 * slot] = make_float4(post[4] * gate[4], post[5] * gate[5], post[6] * gate[6], post[7] * gate[7]);
    }
    auto read_channel = [&](int which, int i, float2 (&w)[4]) {
        const float4 lo = channels[2 * which * slot + i * threads], hi = channels[(2 * which + 1) * slot + i * threads];
        w[0] = make_float2(lo.x, lo.y);
        w[1] = make_float2(lo.z, lo.w);
        w[2] = make_float2(hi.x, hi.y);
        w[3] = make_float2(hi.z, hi.w);
    };
    float2 sum_q[VPT][4], dpre[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum_q[i][j] = dpre[i][j] = both(0.0f);
    // a row's sum of dn * pre_weight * h, and its part of pre_weight's gradient
    auto along_pre = [&](const uint4* from, float pre) {
        float2 s = both(0.0f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i + 1 == VPT && !all) break;
            float2 h[4], g[4], w[4];
            unpack4x2<FP16>(from[kSlotH * slot + i * threads], h);
            unpack4x2<FP16>(from[kSlotDn * slot + i * threads], g);
            read_channel(0, i, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[j] = mul2(g[j], h[j]);
                dpre[i][j] = fused2(g[j], both(pre), dpre[i][j]);
                s = fused2(g[j], w[j], s);
            }
        }
        return s.x + s.y;
    };
    struct Row { float pre, post, gate; };
    auto scalars = [&](int64_t row) {
        Row r{0.0f, 1.0f, 1.0f};
        if (row < a.rows) {
            if (a.pre_weight) r.pre = a.pre_rstd_in[row];
            if (a.post_weight) r.post = a.post_rstd_in[row];
            if (a.gate_kind == EP_GATE_ROW) r.gate = reinterpret_cast<const float*>(a.gate)[row];
        }
        return r;
    };
    Row now = scalars(blockIdx.x);
    copies_wait<STAGES - 1>();
    float2 sums = both(0.0f);
    if (a.pre_weight) sums = row_sums<WARP>(make_float2(along_pre(mine, now.pre), 0.0f), part[1]);
    int parity = 0, stage = 0;
    const uint4* here = mine;   // this row's stage
    int64_t out = blockIdx.x * pitch + at;   // bytes into the gradients
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1, out += gridDim.x * pitch) {
        const Row then = scalars(row + gridDim.x);
        float2 d[VPT][4], s = both(0.0f);
        const float2 pre = both(now.pre), post = both(now.post), gate = both(now.gate), c = both(-sums.x * inv_hidden * now.pre * now.pre);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i + 1 == VPT && !all) break;
            const uint4* from = here + i * threads;
            float2 w[4], x[4];
            if (a.dh) {
                unpack4x2<FP16>(from[kSlotDh * slot], d[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = both(0.0f);
            }
            if (a.pre_weight) {
                unpack4x2<FP16>(from[kSlotH * slot], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = fused2(mul2(x[j], pre), c, d[i][j]);
                unpack4x2<FP16>(from[kSlotDn * slot], x);
                read_channel(0, i, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = fused2(mul2(x[j], w[j]), pre, d[i][j]);
            }
            if (a.dresidual) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = mul2(both(a.residual_scale), d[i][j]);
                st_v4(a.dresidual + out + i * next_vector, pack4x2<FP16>(x));
            }
            float2 v[4];
            unpack4x2<FP16>(from[kSlotY * slot], v);
            read_channel(1, i, w);
            if (element) {
                float2 e[4];
                unpack4x2<FP16>(from[kSlotGate * slot], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = mul2(v[j], post);
                    const float2 q = mul2(d[i][j], v[j]);
                    e[j] = mul2(q, w[j]);
                    sum_q[i][j] = fused2(q, x[j], sum_q[i][j]);
                    d[i][j] = mul2(mul2(d[i][j], w[j]), x[j]);
                    s = fused2(d[i][j], v[j], s);
                }
                st_v4(a.dgate_element + out + i * next_vector, pack4x2<FP16>(e));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = mul2(v[j], post);
                    sum_q[i][j] = fused2(mul2(d[i][j], v[j]), gate, sum_q[i][j]);
                    d[i][j] = mul2(d[i][j], w[j]);
                    s = fused2(d[i][j], v[j], s);
                }
            }
        }
        const uint4* after = stage + 1 == STAGES ? mine : here + slots * slot;
        copies_wait<STAGES - 2>();
        sums = make_float2(a.pre_weight && row + gridDim.x < a.rows ? along_pre(after, then.pre) : 0.0f, s.x + s.y);
        if (a.pre_weight || a.post_weight || a.gate_kind == EP_GATE_ROW) sums = row_sums<WARP>(sums, part[parity]);
        if (a.gate_kind == EP_GATE_ROW && t == 0) a.dgate_row[row] = sums.y;
        const float2 mean = both(-sums.y * inv_hidden), scale = both(now.post * now.gate);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i + 1 == VPT && !all) break;
            if (a.post_weight) {
                float2 v[4];
                unpack4x2<FP16>(here[kSlotY * slot + i * threads], v);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = fused2(mul2(v[j], post), mean, d[i][j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][j] = mul2(d[i][j], scale);
            st_v4(a.dy + out + i * next_vector, pack4x2<FP16>(d[i]));
        }
        fetch(stage);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        here = after;
        now = then;
    }
    // each sum times what it lacks: one of the channels' two factors, or nothing
    auto leave = [&](const float2 (&s)[VPT][4], int which, const void* factor, int fp32) {
        float* to = a.partial + ((int64_t)blockIdx.x * 3 + which) * a.hidden;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i + 1 == VPT && !all) break;
            const int v = i * threads + t;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 1.0f;
            if (factor) load_channels<FP16>(factor, fp32, v, f);
            float4* p = reinterpret_cast<float4*>(to + 8 * v);
            p[0] = make_float4(s[i][0].x * f[0], s[i][0].y * f[1], s[i][1].x * f[2], s[i][1].y * f[3]);
            p[1] = make_float4(s[i][2].x * f[4], s[i][2].y * f[5], s[i][3].x * f[6], s[i][3].y * f[7]);
        }
    };
    const bool channel = a.gate_kind == EP_GATE_CHANNEL;
    if (a.post_weight) leave(sum_q, 0, channel ? a.gate : nullptr, a.gate_fp32);
    if (channel) leave(sum_q, 1, a.post_weight, a.post_fp32);
    if (a.pre_weight) leave(dpre, 2, nullptr, 0);
}

// ---- wider rows: a CTA per row, VPT vectors of 8 columns per thread.  Nothing of the next row is on its way while a row's sums
// are made, and the 84 or 128 registers of 512 threads leave an SM one CTA: 8192 rows of 16384 take 266 us (158 by bytes) and,
// with codes, 309 (139); of 32768, with codes, 747 (279).
template <bool FP16, int VPT>
__global__ void __launch_bounds__(kJoinMaxThreads) ep_join_wide_kernel(const JoinArgs a)
{
    __shared__ float part[2][32];
    const int t = threadIdx.x, stride = blockDim.x;
    const int64_t row = blockIdx.x;
    follow_predecessor();
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
        sum = row_sums<false>(make_float2(sum, 0.0f), part[0]).x;
        const float rstd = root_of(sum / (float)a.hidden + a.eps);
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
    sum = row_sums<false>(make_float2(sum, 0.0f), part[1]).x;
    const float rstd = root_of(sum / (float)a.hidden + a.eps);
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
        const float scale = quick_block_scale(m), inv = quick_reciprocal(scale);   // as above: one rule at every width
        if (in) {
            const uint2 q = make_uint2(e4m3x4_near(f[i][0], f[i][1], f[i][2], f[i][3], scale, inv),
                                       e4m3x4_near(f[i][4], f[i][5], f[i][6], f[i][7], scale, inv));
            *reinterpret_cast<uint2*>(a.q + (row * a.vecs + v) * 8) = q;
            if ((v & 15) == 0) a.scales[row * a.blocks + (v >> 4)] = scale;
        }
    }
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

// Shared memory of a CTA of the team kernels, and how many CTAs an SM holds.
constexpr size_t kJoinShared = 227 * 1024 - 1024;   // less the static part, 256 bytes

int team_vectors(int hidden) { return hidden <= 256 ? 1 : 2; }   // of a thread

int team_threads(int hidden)
{
    const int columns = 8 * team_vectors(hidden);
    return (hidden / columns + (hidden % columns != 0) + 31) / 32 * 32;
}

size_t team_shared(const JoinArgs& a, int stages, int slots)
{
    return (size_t)(stages * slots + channel_vectors(a)) * team_vectors(a.hidden) * team_threads(a.hidden) * 16;
}

int team_ctas_per_sm(int most_threads, int threads, size_t shared)
{
    const int by_threads = most_threads / threads, by_shared = (int)(228 * 1024 / (shared + 2048));
    const int n = by_threads < by_shared ? by_threads : by_shared;
    return n < 1 ? 1 : n > 24 ? 24 : n;
}

template <auto* K>
cudaError_t launch_team(const JoinArgs& a, int64_t ctas, size_t shared, cudaStream_t s)
{
    const cudaError_t e = allow_all_shared<K>();
    return e != cudaSuccess ? e : launch_dependent(K, dim3((unsigned)ctas), dim3(team_threads(a.hidden)), shared, s, a);
}

template <bool FP16>
cudaError_t launch_join(const JoinArgs& a, int sms, cudaStream_t s)
{
    if (a.hidden > kJoinTeamHidden) {
        const int vpt = a.vecs <= 4 * kJoinMaxThreads ? 4 : 8;
        const dim3 grid((unsigned)a.rows), block(((a.vecs + vpt - 1) / vpt + 31) / 32 * 32);
        if (vpt == 4) return launch_dependent(ep_join_wide_kernel<FP16, 4>, grid, block, 0, s, a);
        return launch_dependent(ep_join_wide_kernel<FP16, 8>, grid, block, 0, s, a);
    }
    // Four stages where they leave an SM as many CTAs as its registers do, else two: two CTAs on an SM hide each other's
    // barriers.
    const int threads = team_threads(a.hidden), slots = a.gate_kind == EP_GATE_ELEMENT ? 3 : 2;
    constexpr int kThreads = 2 * kJoinTeamThreads;
    // one launch for each number of stages, so that the shared memory is that of the kernel's own
    auto launch = [&](auto* kernel_of, int stages) {
        const size_t shared = team_shared(a, stages, slots);
        const int64_t fit = (int64_t)sms * team_ctas_per_sm(kThreads, threads, shared);
        return kernel_of(a, a.rows < fit ? a.rows : fit, shared, s);
    };
    if (a.hidden <= 256) return launch(&launch_team<ep_join_team_kernel<FP16, true, 1, 4>>, 4);
    if (threads == 32) return launch(&launch_team<ep_join_team_kernel<FP16, true, 2, 4>>, 4);
    const size_t shared = team_shared(a, 4, slots);
    if (shared <= kJoinShared && team_ctas_per_sm(kThreads, threads, shared) == team_ctas_per_sm(kThreads, threads, 0))
        return launch(&launch_team<ep_join_team_kernel<FP16, false, 2, 4>>, 4);
    return launch(&launch_team<ep_join_team_kernel<FP16, false, 2, 2>>, 2);
}

// CTAs of the gradient's kernel, by the shape alone, because they fix the order of the sums: as many as the SMs hold with
// the most shared memory that a CTA of this width may take, but no fewer than kRowsPerCta rows to each while that leaves
// every SM one, because every CTA leaves three rows of sums.
constexpr int kRowsPerCta = 4;

int join_backward_ctas(int64_t rows, int hidden, int sms)
{
    const int threads = team_threads(hidden);
    const int64_t fit = (int64_t)sms * team_ctas_per_sm(kJoinTeamThreads, threads, (size_t)(3 * 5 + kBackChannels) * team_vectors(hidden) * threads * 16);
    const int64_t want = (rows + kRowsPerCta - 1) / kRowsPerCta;
    const int64_t least = rows < sms ? rows : sms;
    return (int)(want < least ? least : want < fit ? want : fit);
}

template <bool FP16>
cudaError_t launch_join_backward(const JoinArgs& a, int ctas, cudaStream_t s)
{
    const int slots = a.gate_kind == EP_GATE_ELEMENT ? 5 : 4;
    auto shared = [&](int stages) { return (size_t)(stages * slots + kBackChannels) * team_vectors(a.hidden) * team_threads(a.hidden) * 16; };
    if (a.hidden <= 256) return launch_team<ep_join_backward_kernel<FP16, true, 1, 3>>(a, ctas, shared(3), s);
    if (team_threads(a.hidden) == 32) return launch_team<ep_join_backward_kernel<FP16, true, 2, 3>>(a, ctas, shared(3), s);
    if (shared(3) <= kJoinShared) return launch_team<ep_join_backward_kernel<FP16, false, 2, 3>>(a, ctas, shared(3), s);
    return launch_team<ep_join_backward_kernel<FP16, false, 2, 2>>(a, ctas, shared(2), s);
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
    const int sms = layer_num_sms();
    if (sms == 0) return layer_fail(EP_ERR_CUDA, "%s: cannot tell the current device's multiprocessors", who);
    const cudaError_t e = fp16 ? launch_join<true>(a, sms, s) : launch_join<false>(a, sms, s);
    return layer_cuda(e, "ep_rms_norm_join: launch");
}

extern "C" size_t ep_rms_norm_join_workspace_bytes(int64_t rows, int hidden)
{
    using namespace ep;
    if (rows <= 0 || rows >= (int64_t)1 << 31 || hidden < 16 || hidden > kJoinTeamHidden || hidden % 16 != 0) return 0;
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
    if (int rc = check_join(who, join, kJoinTeamHidden, a)) return rc;
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
