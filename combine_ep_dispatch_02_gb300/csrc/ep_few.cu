// ep_few.cu -- a whole mixture-of-experts layer for a few rows, in two kernels.
//
//   [gate; up] = up[e] x,  z = gate * sigmoid(gate) * up,  out[row] = sum over the row's experts e, ascending, of
//   weight * down[e] z
//
// with e4m3 weights and one FP32 scale per 128 x 128 block.  The time is that of reading the weights of the experts
// that any row names, once: 3 * inner * hidden bytes each.  So a warp reads 16 or 32 of their rows, 128 columns a step,
// through a ring of its own in shared memory that only its own lanes' copies fill and read, a few steps ahead: it meets
// no barrier on the way, and so few rows spread any layer over the SMs.
//
// Measured, with 8 experts of 32 of 7168 x 2048: one row 64 us (352 MB, 5.5 TB/s; 52 by bytes), with 20 of 32 for 4 rows
// 154 us (5.7 TB/s).  Each further expert takes 7.3 us, 0.90 of a copy's bandwidth; some 6 us are the two kernels' sorts, first
// trips to memory and last steps.  From two rows to an expert on the matrix instructions of 16 x 8 (and what makes their
// second operand) bound it: 16 rows of 8 experts of 32 take 252 us, 64 rows 469.  One BF16 row, whose values take a
// multiplication and a conversion each, 2 us more than one of e4m3 or FP16; 64 of them, on 32 of 256 experts, 231 us for 222.
//
// A lane's 16 bytes are 16 columns of one row.  Which of the K columns share a matrix instruction is free, as long as
// both operands agree; so a lane takes its own 16 for four instructions and reads the same 16 of the other operand's
// row.  Codes become FP16 on the way, which is exact; the sums of a block of 128 are FP32 and enter the row's, times
// the scales, in FP32.
//
// Each CTA finds by itself what it has to do: it sorts the rows by expert, in shared memory, by a bit for each row and
// expert.  A row that names an expert in several slots counts once, with the sum of those slots' weights.
//
// The first kernel leaves z as FP16 with a power of two for every 8 columns.  The second brings a block of 128 columns to one
// power of two, so that its operand keeps 11 bits down to 2^-28 of the block's largest value, and what is smaller to 2^-39 of
// that value; the e4m3 that a chain of products would leave has 4 bits.  The second kernel's CTA owns 16 output
// columns, over every expert: each output is summed in one place, in a fixed order.  It is a programmatic dependent
// that reads weights before it waits: the first kernel lets it start only after its own wait, when all that precedes the
// call has completed, and the weights are nothing that the first writes.
#include <type_traits>

#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kFewRows = 128;          // rows of a call
constexpr int kFewPairs = 4096;        // (row, slot) pairs of a call
constexpr int kFewExperts = 1024;
constexpr int kUpWarps = 4;            // of a CTA of the first kernel
constexpr uint16_t kNone = 0xFFFF;

enum { kFromE4m3 = 0, kFromFp16 = 1, kFromBf16 = 2, kFromZ = 3 };   // what the rows are held as

struct FewArgs {
    const uint8_t* x;
    const float* x_scales;
    const int32_t* indices;
    const float* weights;
    const uint8_t* up;
    const float* up_scales;
    const uint8_t* down;
    const float* down_scales;
    uint8_t* z;          // [pairs][inner] FP16
    uint8_t* z_exp;      // [pairs][inner / 8]: 128 + the power of two of 8 columns, 0 where all are 0
    void* out;
    int rows, k, pairs, first, experts, H, I;
    int hb, ib, ub;      // 128-blocks of hidden, inner and 2 * inner
    int split;           // warps that share a unit's K in the first kernel: 1, 2 or 4
    int out_fp16;
};

// The rows by expert, in shared memory: entry i holds up to 8 * NT rows of expert[i], list[start[i]] .. list[start[i + 1]
// - 1].  Every CTA makes the same: z lies by place in the list, and a unit's rows are the same whichever CTA works on it.
struct Entries {
    uint16_t *local, *list, *expert, *start;   // [pairs] each, start one more; local: a pair's expert, kNone for none here
    int* cursor;                               // [experts]: place of an expert's first row
    uint32_t* named;                           // [experts][words]: the rows that name an expert, a bit each
    int* count;
};

__host__ __device__ inline int row_words(int rows) { return (rows + 31) / 32; }

__host__ __device__ inline size_t entries_bytes(int pairs, int experts, int rows)
{
    return (size_t)((4 * pairs + 1) * 2 + 15) / 16 * 16 + ((size_t)experts * (1 + row_words(rows)) + 4) / 4 * 16;
}

__device__ __forceinline__ Entries entries_at(uint8_t* p, const FewArgs& a)
{
    Entries s;
    s.local = reinterpret_cast<uint16_t*>(p);
    s.list = s.local + a.pairs;
    s.expert = s.list + a.pairs;
    s.start = s.expert + a.pairs;
    s.cursor = reinterpret_cast<int*>(p + ((4 * a.pairs + 1) * 2 + 15) / 16 * 16);
    s.count = s.cursor + a.experts;
    s.named = reinterpret_cast<uint32_t*>(s.count + 1);
    return s;
}

// 32 bits from where all SMs see the same, not from this SM's cache.
__device__ __forceinline__ int32_t load_shared_view(const int32_t* p)
{
    int32_t v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Place in the list of a row that names expert e.
__device__ __forceinline__ int place_of(const Entries& s, int words, int e, int row)
{
    int at = s.cursor[e] + __popc(s.named[e * words + row / 32] & ((1u << (row & 31)) - 1));
    for (int w = 0; w < row / 32; ++w) at += __popc(s.named[e * words + w]);
    return at;
}

// Sorts the rows into entries of up to `per` rows; returns their number.  All threads of the CTA.
__device__ __forceinline__ int make_entries(const FewArgs& a, const Entries& s, int per)
{
    const int words = row_words(a.rows);
    for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
        const int32_t id = load_shared_view(a.indices + p);
        const int64_t e = (int64_t)id - a.first;
        s.local[p] = id >= 0 && e >= 0 && e < a.experts ? (uint16_t)e : kNone;   // first may be negative, an id here not
    }
    for (int i = threadIdx.x; i < a.experts * words; i += blockDim.x) s.named[i] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
        const int e = s.local[p], row = p / a.k;
        if (e != kNone) atomicOr(&s.named[e * words + row / 32], 1u << (row & 31));
    }
    __syncthreads();
    if (threadIdx.x < 32) {   // exclusive sums of rows (low half) and entries (high half)
        const int lane = threadIdx.x;
        int carry = 0;
        for (int b = 0; b < a.experts; b += 32) {
            const int e = b + lane;
            int rows = 0;
            if (e < a.experts)
                for (int w = 0; w < words; ++w) rows += __popc(s.named[e * words + w]);
            const int n = (rows + per - 1) / per, v = n << 16 | rows;
            int sum = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += u;
            }
            const int at = carry + sum - v, row0 = at & 0xFFFF, entry0 = at >> 16;
            for (int i = 0; i < n; ++i) {
                s.expert[entry0 + i] = (uint16_t)e;
                s.start[entry0 + i] = (uint16_t)(row0 + i * per);
            }
            if (e < a.experts) s.cursor[e] = row0;
            carry += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) {
            s.start[carry >> 16] = (uint16_t)(carry & 0xFFFF);
            *s.count = carry >> 16;
        }
    }
    __syncthreads();
    for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
        const int e = s.local[p], row = p / a.k;
        if (e == kNone) continue;
        s.list[place_of(s, words, e, row)] = (uint16_t)row;   // slots of a row that name one expert write the same
    }
    __syncthreads();
    return *s.count;
}

// 16 bytes of weights on their way into shared memory, past this SM's cache; zeros if not `in`.
__device__ __forceinline__ void copy_weights(uint32_t to, const uint8_t* from, bool in)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" :: "r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}

// A step's 16 rows of weights, a lane's 16 bytes of four: rows g and g + 8, then the second 64 columns of both.
__device__ __forceinline__ void read_weights(uint32_t from, uint4 (&w)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w) : "r"(from + 512 * i) : "memory");
}

// Two e4m3 codes to two FP16 values, exactly; the low or the high half of w.
__device__ __forceinline__ uint32_t half_codes(uint32_t w, bool high)
{
    uint32_t r;
    if (high) asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
    else asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^n for n in -126..127.
__device__ __forceinline__ float power2(int n) { return __int_as_float((n + 127) << 23); }

// 2^-m and 2^-n as FP16 in the low and the high half, held at its smallest number, 2^-24; m, n >= 0.
__device__ __forceinline__ uint32_t half_power2(int m, int n)
{
    return pack2<true>(power2(-min(m, 24)), power2(-min(n, 24)));
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// A lane's part of the other operand over a block of 128 columns, as it lies in memory: columns 16 q .. + 15 of both
// 64-column chunks of a row, and what it takes to make FP16 values of them.
template <int FROM>
struct Rows16 {
    uint4 v[FROM == kFromE4m3 ? 2 : 4];
    uint32_t e0, e1;   // kFromZ: the powers of two of either chunk's 8 + 8 columns
    float f;           // kFromE4m3: the block's scale
};

// at: bytes from x (or z) to the lane's columns; scale: elements from x_scales (bytes from z_exp) to the block's.  WHOLE: all
// columns exist; otherwise, of a short last block, whose weights read as zeros, those of in0 and in1.
template <int FROM, bool WHOLE>
__device__ __forceinline__ void fetch_rows(const FewArgs& a, uint32_t at, uint32_t scale, bool in0, bool in1, Rows16<FROM>& r)
{
    const uint4* p = reinterpret_cast<const uint4*>((FROM == kFromZ ? a.z : a.x) + at);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (FROM == kFromE4m3) {
        r.v[0] = WHOLE || in0 ? p[0] : zero;
        r.v[1] = WHOLE || in1 ? p[4] : zero;
        r.f = a.x_scales[scale];
    } else {
        r.v[0] = WHOLE || in0 ? p[0] : zero;
        r.v[1] = WHOLE || in0 ? p[1] : zero;
        r.v[2] = WHOLE || in1 ? p[8] : zero;
        r.v[3] = WHOLE || in1 ? p[9] : zero;
        if constexpr (FROM == kFromZ) {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(a.z_exp + scale);
            r.e0 = WHOLE || in0 ? e[0] : 0;
            r.e1 = WHOLE || in1 ? e[4] : 0;
        }
    }
}

// The same as FP16; returns the factor that the block's sums take for that row.
template <int FROM>
__device__ __forceinline__ float half_rows(const Rows16<FROM>& r, uint32_t (&b)[16])
{
    if constexpr (FROM == kFromE4m3) {
        const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            b[2 * i] = half_codes(w[i], false);
            b[2 * i + 1] = half_codes(w[i], true);
        }
        return r.f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[4 * i] = r.v[i].x;
            b[4 * i + 1] = r.v[i].y;
            b[4 * i + 2] = r.v[i].z;
            b[4 * i + 3] = r.v[i].w;
        }
        if constexpr (FROM == kFromFp16) return 1.0f;
        if constexpr (FROM == kFromZ) {
            // Each 8 columns to the largest power of two of the block's, which lies in 2^14 .. 2^15.  Below FP16's normal
            // numbers, 2^-28 of it, bits are lost: 2^-39 of it at the most, and half as much in the first of two steps.
            const int e[4] = {(int)(r.e0 & 0xFF), (int)(r.e0 >> 8), (int)(r.e1 & 0xFF), (int)(r.e1 >> 8)};
            int top = max(max(e[0], e[1]), max(e[2], e[3]));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            auto bring = [&](int i, uint32_t f) {   // the lane's vectors i and i + 1
                const uint32_t lo = __byte_perm(f, 0, 0x1010), hi = __byte_perm(f, 0, 0x3232);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[4 * i + j] = mul_half2(b[4 * i + j], lo);
                    b[4 * i + 4 + j] = mul_half2(b[4 * i + 4 + j], hi);
                }
            };
            const uint32_t f0 = half_power2(top - e[0], top - e[1]), f1 = half_power2(top - e[2], top - e[3]);
            bring(0, f0);
            bring(2, f1);
            // At 2^-24, of all powers the one with the lowest bit, the way may go on: rare, and nothing is left past 2^-48.
            if ((f0 | f1) & 0x00010001u) {
                bring(0, half_power2(max(top - e[0] - 24, 0), max(top - e[1] - 24, 0)));
                bring(2, half_power2(max(top - e[2] - 24, 0), max(top - e[3] - 24, 0)));
            }
            return power2(max(top, 18) - 142);
        }
        if constexpr (FROM == kFromBf16) {
            // BF16's 8 bits fit FP16's 11; its range does not, so the block's largest value is brought to 2^14 .. 2^15
            uint32_t top = 0;   // of the magnitudes' bits, two at a time
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __vmaxu2(top, b[i] & 0x7FFF7FFFu);
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(max((int)(top >> 7) - 127, -110), 126);
            const float f = power2(14 - e);
#pragma unroll
            for (int i = 0; i < 16; ++i) b[i] = pack2<true>(bf16_lo(b[i]) * f, bf16_hi(b[i]) * f);
            return power2(e - 14);
        }
    }
    return 0.0f;
}

constexpr int kStepBytes = 2048;   // 16 rows of a block of 128 columns

// Eight columns' sums of a block of 128, times their scales, into tot: w holds the block's 16 rows of weights (row g,
// row g + 8; then the second 64 columns), f the lane's row's factor (1 unless FACTOR), s0 and s1 the scales of rows g and
// g + 8.
template <bool FACTOR>
__device__ __forceinline__ void add_block(float (&tot)[4], const uint4 (&w)[4], const uint32_t (&b)[16], float f, float s0,
                                          float s1)
{
    float d[2][4] = {};   // two sums, so that only four products wait for one another
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t lo = m == 0 ? w[2 * c].x : m == 1 ? w[2 * c].y : m == 2 ? w[2 * c].z : w[2 * c].w;
            const uint32_t hi = m == 0 ? w[2 * c + 1].x : m == 1 ? w[2 * c + 1].y : m == 2 ? w[2 * c + 1].z : w[2 * c + 1].w;
            const uint32_t x[4] = {half_codes(lo, false), half_codes(hi, false), half_codes(lo, true), half_codes(hi, true)};
            mma_f16(d[c], x, b[8 * c + 2 * m], b[8 * c + 2 * m + 1]);
        }
    }
    float f0 = 1.0f, f1 = 1.0f;
    if constexpr (FACTOR) {
        const int q = threadIdx.x & 3;
        f0 = __shfl_sync(0xffffffffu, f, 8 * q);
        f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);
    }
    tot[0] = fmaf(d[0][0] + d[1][0], s0 * f0, tot[0]);
    tot[1] = fmaf(d[0][1] + d[1][1], s0 * f1, tot[1]);
    tot[2] = fmaf(d[0][2] + d[1][2], s1 * f0, tot[2]);
    tot[3] = fmaf(d[0][3] + d[1][3], s1 * f1, tot[3]);
}

// Two matrices' sums of a block at once; their weights, from `from` in shared memory on, are read one after the other.
template <bool FACTOR>
__device__ __forceinline__ void add_two_blocks(float (&tot)[2][4], uint32_t from, const uint32_t (&b)[16], float f, float s0,
                                               float s1)
{
    float f0 = 1.0f, f1 = 1.0f;
    if constexpr (FACTOR) {
        const int q = threadIdx.x & 3;
        f0 = __shfl_sync(0xffffffffu, f, 8 * q);
        f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);
    }
    const float scale[4] = {s0 * f0, s0 * f1, s1 * f0, s1 * f1};
    uint4 w[2][4];
    read_weights(from, w[0]);
    read_weights(from + kStepBytes, w[1]);
    float d[2][4] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint4 &l = w[m][2 * c], &h = w[m][2 * c + 1];
                const uint32_t lo = i == 0 ? l.x : i == 1 ? l.y : i == 2 ? l.z : l.w, hi = i == 0 ? h.x : i == 1 ? h.y : i == 2 ? h.z : h.w;
                const uint32_t x[4] = {half_codes(lo, false), half_codes(hi, false), half_codes(lo, true), half_codes(hi, true)};
                mma_f16(d[m], x, b[8 * c + 2 * i], b[8 * c + 2 * i + 1]);
            }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[m][i] = fmaf(d[m][i], scale[i], tot[m][i]);
}

// Steps that a warp's weights are read ahead, of 4 KB in the first kernel and 2 KB in the second; the other operand and the
// scales are read one step ahead.  More of them took longer: 7 rows of 8 experts of 7168 x 2048 194 us, with 3 and 6 steps
// 261 us, because what shared memory takes the other operand lacks in the SM's cache.
constexpr int kUpStepBytes = 2 * kStepBytes, kUpAhead = 2, kDownAhead = 3;

// Warps of an SM, by the registers that they take.
template <int NT>
constexpr int kUpWarpsPerSm = NT == 1 ? 16 : 12;
template <int NT>
constexpr int kDownWarpsPerSm = NT == 1 ? 20 : 16;

// Up projection and SwiGLU.  A unit is 16 columns of z for one entry, two matrices of 8 gate rows and 8 up rows, so that what
// it takes to make the other operand is shared by two; a unit is a warp's, or with SPLIT `split` warps', which share its K.
template <int FROM, int NT, bool SPLIT>
__global__ void __launch_bounds__(32 * kUpWarps, kUpWarpsPerSm<NT> / kUpWarps) ep_few_up_kernel(const FewArgs a)
{
    extern __shared__ __align__(16) uint8_t shared[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const Entries s = entries_at(shared, a);
    follow_predecessor();
    const int entries = make_entries(a, s, 8 * NT);
    const int split = SPLIT ? a.split : 1, teams = kUpWarps / split, team = warp / split, member = warp % split;
    const int slices = a.I / 16, units = entries * slices;
    const int k_lo = a.hb * member / split, k_hi = a.hb * (member + 1) / split, nb = k_hi - k_lo;
    const int u0 = blockIdx.x * teams + team, stride = gridDim.x * teams;
    const int mine = u0 < units ? (units - 1 - u0) / stride + 1 : 0;
    const int steps = mine * nb;

    constexpr int D = kUpAhead, kElement = FROM == kFromE4m3 ? 1 : 2;
    constexpr bool kFactor = FROM != kFromFp16;
    // a lane fills and reads its own bytes of the warp's ring, so that nothing passes between lanes
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(shared + entries_bytes(a.pairs, a.experts, a.rows)) +
                          warp * D * kUpStepBytes + 16 * lane;
    const uint32_t ring_end = ring + D * kUpStepBytes;
    // Of K's last block a lane's columns of either chunk may not exist.
    const bool tail = a.H % 128 != 0 && k_hi == a.hb, tail0 = !tail || 128 * (a.hb - 1) + 16 * q < a.H,
               tail1 = !tail || 128 * (a.hb - 1) + 16 * q + 64 < a.H;
    const int whole = a.H / 128;   // blocks without such columns
    const int64_t up_rows = (int64_t)a.I * a.H, eight_rows = 8 * (int64_t)a.H;
    int lu = u0, left = steps > 0 ? nb : 0;   // of the loads: unit, and its blocks not yet under way
    const uint8_t *lp = nullptr, *lq = nullptr;
    auto point = [&] {
        const int entry = lu / slices;
        lp = a.up + ((int64_t)s.expert[entry] * 2 * a.I + 16 * (lu - entry * slices) + g) * a.H + 128 * k_lo + 16 * q;
        lq = lp + up_rows;
    };
    if (left > 0) point();
    auto load = [&](uint32_t to) {
        if (left > 0) {
            const bool in0 = left > 1 || tail0, in1 = left > 1 || tail1;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint8_t *p = lp + m * eight_rows, *r = lq + m * eight_rows;
                copy_weights(to + kStepBytes * m, p, in0);
                copy_weights(to + kStepBytes * m + 512, r, in0);
                copy_weights(to + kStepBytes * m + 1024, p + 64, in1);
                copy_weights(to + kStepBytes * m + 1536, r + 64, in1);
            }
            lp += 128;
            lq += 128;
            if (--left == 0) {
                lu += stride;
                if (lu < units) {
                    left = nb;
                    point();
                }
            }
        }
        copies_commit();
    };
    for (uint32_t to = ring; to != ring_end; to += kUpStepBytes) load(to);

    // the unit whose operand is fetched, and the block of K.  Columns past an entry's rows repeat one of its rows: what
    // they sum up is not used.
    int u = u0, k = k_lo, first = 0, n = 0, slice = 0;
    uint32_t row_at[NT], row_scale[NT];
    const float *gs = nullptr, *us = nullptr;   // the unit's scales
    auto begin = [&] {
        const int entry = u / slices;
        slice = u - entry * slices;
        first = s.start[entry];
        n = s.start[entry + 1] - first;
        const float* es = a.up_scales + (int64_t)s.expert[entry] * a.ub * a.hb;
        gs = es + (int64_t)(16 * slice / 128) * a.hb;
        us = es + (int64_t)((a.I + 16 * slice) / 128) * a.hb;
        k = k_lo;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t row = s.list[first + (8 * t + g < n ? 8 * t + g : 0)];
            row_at[t] = (row * a.H + 16 * q) * kElement;
            row_scale[t] = row * a.hb;
        }
    };
    Rows16<FROM> x[NT];
    float s0 = 0.0f, s1 = 0.0f, tot[NT][2][4];
    auto fetch = [&](int t, Rows16<FROM>& r) {
        const uint32_t at = row_at[t] + 128 * kElement * k, scale = row_scale[t] + k;
        if (k < whole) fetch_rows<FROM, true>(a, at, scale, true, true, r);
        else fetch_rows<FROM, false>(a, at, scale, tail0, tail1, r);
    };
    auto scales = [&] {
        s0 = gs[k];
        s1 = us[k];
    };
    auto clear = [&] {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) tot[t][i / 4][i & 3] = 0.0f;
    };
    clear();
    if (steps > 0) {
        begin();
        scales();
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (8 * t < n) fetch(t, x[t]);
    }
    // z of a unit from its whole sums, and its power of two
    auto finish = [&](int first, int n, int slice) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= n) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = i / 2, c = i & 1;
                const float z = tot[t][m][c] * sigmoid_and_rest(tot[t][m][c]).x * tot[t][m][2 + c];
                float top = fmaxf(fabsf(z), 0.0f);   // NaN counts as 0
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // the largest of the 8 to 2^14 .. 2^15; an infinity stays one
                const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -110), 127);
                const int column = 8 * t + 2 * q + c;
                if (column >= n) continue;
                const int64_t place = first + column;
                reinterpret_cast<__half*>(a.z)[place * a.I + 16 * slice + 8 * m + g] = __float2half_rn(z * power2(14 - e));
                if (g == 0) a.z_exp[place * 2 * slices + 2 * slice + m] = top > 0.0f ? (uint8_t)(e + 128) : 0;
            }
        }
    };
    uint32_t at = ring;
    // One step of a unit of `rows` rows, whose operand is here.  The next step's is fetched: that of
    // the same unit's next block, or, once `next` has begun another unit, of its first.  MORE: there is a next step.
    auto step = [&](auto more, int rows, auto next) {
        constexpr bool MORE = decltype(more)::value;
        copies_wait<D - 1>();
        const float s0_now = s0, s1_now = s1;
        if constexpr (MORE) {
            next();
            scales();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= rows && (!MORE || 8 * t >= n)) break;
            uint32_t b[16];
            const float f = half_rows<FROM>(x[t], b);   // of nothing, past `rows`: not used
            if (MORE && 8 * t < n) fetch(t, x[t]);
            if (8 * t < rows) add_two_blocks<kFactor>(tot[t], at, b, f, s0_now, s1_now);
        }
        load(at);   // its bytes have been read, and used
        at = at + kUpStepBytes == ring_end ? ring : at + kUpStepBytes;
    };
    constexpr std::true_type kMore{};
    constexpr std::false_type kLast{};
    // a unit from its first step to its last, during which the next unit's first operand is fetched
    auto unit_steps = [&](bool another) {
        const int rows = n;
        for (int i = 1; i < nb; ++i) step(kMore, rows, [&] { ++k; });
        if (another) step(kMore, rows, [&] { u += stride; begin(); });
        else step(kLast, rows, [] {});
    };
    if constexpr (!SPLIT) {
        for (int i = 1; i <= mine; ++i) {
            const int first_now = first, n_now = n, slice_now = slice;
            unit_steps(i < mine);
            finish(first_now, n_now, slice_now);
            clear();
        }
        return;
    }
    // a unit's warps meet once per round, and every team of the CTA makes as many rounds
    __shared__ float4 parts[kUpWarps][NT][2][32];   // sums of a unit's K
    const int first_unit = blockIdx.x * teams;
    const int rounds = first_unit < units ? (units - 1 - first_unit) / stride + 1 : 0;
    for (int round = 0; round < rounds; ++round) {
        const int unit = u0 + round * stride;
        const bool has = unit < units;
        const int entry = has ? unit / slices : 0, slice_now = unit - entry * slices;
        const int first_now = has ? s.start[entry] : 0, n_now = has ? s.start[entry + 1] - first_now : 0;
        if (has && nb > 0) unit_steps(round + 1 < mine);
        if (member > 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    if (8 * t < n_now)
                        parts[warp][t][m][lane] = make_float4(tot[t][m][0], tot[t][m][1], tot[t][m][2], tot[t][m][3]);
        }
        __syncthreads();
        if (member == 0 && has) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (8 * t >= n_now) break;
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    for (int w = 1; w < split; ++w) {
                        const float4 v = parts[warp + w][t][m][lane];
                        tot[t][m][0] += v.x;
                        tot[t][m][1] += v.y;
                        tot[t][m][2] += v.z;
                        tot[t][m][3] += v.w;
                    }
            }
            finish(first_now, n_now, slice_now);
        }
        __syncthreads();   // the sums have been taken
        clear();
    }
}

// Down projection and the weighted sum.  A CTA owns 16 output columns; its warps share the blocks of all entries' K
// evenly, and each keeps the rows' sums of its own part in shared memory.
template <int NT>
__global__ void __launch_bounds__(32 * kDownWarpsPerSm<NT>) ep_few_down_kernel(const FewArgs a)
{
    extern __shared__ __align__(16) uint8_t shared[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int warps = blockDim.x >> 5, h0 = 16 * blockIdx.x;
    const Entries s = entries_at(shared, a);
    float* share = reinterpret_cast<float*>(shared + entries_bytes(a.pairs, a.experts, a.rows));   // [pairs]: weights by list place
    float* sums = share + (a.pairs + 3) / 4 * 4;                                           // [warps][rows][16]
    // Before its wait this kernel reads what the one before it does not write, and that has let it start only after its
    // own wait, when all that precedes the call had reached L2: ids and their weights past this SM's cache, which may hold
    // what was there before, and the experts' weights.
    const int entries = make_entries(a, s, 8 * NT);
    const int total = entries * a.ib;
    const int lo = (int)((int64_t)total * warp / warps), hi = (int)((int64_t)total * (warp + 1) / warps);

    constexpr int D = kDownAhead;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sums + (size_t)warps * a.rows * 16) + warp * D * kStepBytes + 16 * lane;
    const uint32_t ring_end = ring + D * kStepBytes;
    // Of K's last block a lane's columns of either chunk may not exist.
    const bool tail0 = 128 * (a.ib - 1) + 16 * q < a.I, tail1 = 128 * (a.ib - 1) + 16 * q + 64 < a.I;
    const int whole = a.I / 128;   // blocks without such columns
    const int64_t eight_rows = 8 * (int64_t)a.I;
    int lb = lo, le = lo / a.ib, left = a.ib - (lo - le * a.ib);   // of the loads: block, its entry, the entry's blocks left
    const uint8_t* lp = nullptr;
    auto point = [&] { lp = a.down + ((int64_t)s.expert[le] * a.H + h0 + g) * a.I + 128 * (a.ib - left) + 16 * q; };
    if (lb < hi) point();
    auto load = [&](uint32_t to) {
        if (lb < hi) {
            const bool in0 = left > 1 || tail0, in1 = left > 1 || tail1;
            copy_weights(to, lp, in0);
            copy_weights(to + 512, lp + eight_rows, in0);
            copy_weights(to + 1024, lp + 64, in1);
            copy_weights(to + 1536, lp + eight_rows + 64, in1);
            ++lb;
            lp += 128;
            if (--left == 0) {
                left = a.ib;
                ++le;
                if (lb < hi) point();
            }
        }
        copies_commit();
    };
    for (uint32_t to = ring; to != ring_end; to += kStepBytes) load(to);
    for (int i = threadIdx.x; i < warps * a.rows * 16; i += blockDim.x) sums[i] = 0.0f;
    for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
        const int e = s.local[p], row = p / a.k;
        if (e == kNone) continue;
        float w = 0.0f;
        for (int j = row * a.k; j < (row + 1) * a.k; ++j)
            if (s.local[j] == e) w += __int_as_float(load_shared_view(reinterpret_cast<const int32_t*>(a.weights) + j));
        share[place_of(s, row_words(a.rows), e, row)] = w;
    }
    __syncthreads();
    follow_predecessor();

    float* own = sums + warp * a.rows * 16;
    // the entry whose operand is fetched, and the block of K; columns past an entry's rows as in the first kernel
    int e = lo / a.ib, k = lo - e * a.ib, first = 0, n = 0;
    uint32_t row_at[NT], row_exp[NT];
    const float* ds = nullptr;
    auto begin = [&] {
        first = s.start[e];
        n = s.start[e + 1] - first;
        ds = a.down_scales + ((int64_t)s.expert[e] * a.hb + h0 / 128) * a.ib;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t place = first + (8 * t + g < n ? 8 * t + g : 0);
            row_at[t] = (place * a.I + 16 * q) * 2;
            row_exp[t] = place * (a.I / 8) + 2 * q;
        }
    };
    Rows16<kFromZ> x[NT];
    float sc = 0.0f, tot[NT][4];
    auto fetch = [&](int t, Rows16<kFromZ>& r) {
        const uint32_t at = row_at[t] + 256 * k, exp = row_exp[t] + 16 * k;
        if (k < whole) fetch_rows<kFromZ, true>(a, at, exp, true, true, r);
        else fetch_rows<kFromZ, false>(a, at, exp, tail0, tail1, r);
    };
    auto clear = [&] {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[t][i] = 0.0f;
    };
    clear();
    if (lo < hi) {
        begin();
        sc = ds[k];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (8 * t < n) fetch(t, x[t]);
    }
    // an entry's rows are distinct, so that no two lanes add to one place
    auto finish = [&](int first, int n) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= n) break;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int column = 8 * t + 2 * q + c;
                if (column >= n) continue;
                const float w = share[first + column];
                float* to = own + s.list[first + column] * 16 + g;
                to[0] = fmaf(w, tot[t][c], to[0]);
                to[8] = fmaf(w, tot[t][2 + c], to[8]);
            }
        }
        __syncwarp();
    };
    uint32_t at = ring;
    auto step = [&](auto more, int rows, auto next) {   // as in the first kernel
        constexpr bool MORE = decltype(more)::value;
        uint4 w[4];
        copies_wait<D - 1>();
        read_weights(at, w);
        const float sc_now = sc;
        if constexpr (MORE) {
            next();
            sc = ds[k];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= rows && (!MORE || 8 * t >= n)) break;
            uint32_t b[16];
            const float f = half_rows<kFromZ>(x[t], b);   // of nothing, past `rows`: not used
            if (MORE && 8 * t < n) fetch(t, x[t]);
            if (8 * t < rows) add_block<true>(tot[t], w, b, f, sc_now, sc_now);
        }
        load(at);   // its bytes are in registers, and used
        at = at + kStepBytes == ring_end ? ring : at + kStepBytes;
    };
    constexpr std::true_type kMore{};
    constexpr std::false_type kLast{};
    for (int i = lo; i < hi;) {   // an entry, or what of its K is this warp's
        const int first_now = first, n_now = n, blocks = min(a.ib - k, hi - i);
        for (int j = 1; j < blocks; ++j) step(kMore, n_now, [&] { ++k; });
        i += blocks;
        if (i < hi) step(kMore, n_now, [&] { ++e; k = 0; begin(); });
        else step(kLast, n_now, [] {});
        finish(first_now, n_now);
        clear();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.rows * 16; i += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < warps; ++w) v += sums[w * a.rows * 16 + i];
        const int64_t at = (int64_t)(i / 16) * a.H + h0 + (i & 15);
        if (a.out_fp16) reinterpret_cast<__half*>(a.out)[at] = __float2half_rn(v);
        else reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    }
}

template <int FROM, int NT>
cudaError_t launch_up(const FewArgs& a, int sms, cudaStream_t s)
{
    const size_t shared = entries_bytes(a.pairs, a.experts, a.rows) + (size_t)kUpWarps * kUpAhead * kUpStepBytes;
    const int64_t entries = a.pairs < a.experts ? a.pairs : (int64_t)a.experts + a.pairs / (8 * NT);   // at most
    const int64_t teams = kUpWarps / a.split, ctas = (entries * (a.I / 16) + teams - 1) / teams;
    const int64_t fit = (int64_t)sms * (kUpWarpsPerSm<NT> / kUpWarps);
    const dim3 grid((unsigned)(ctas < fit ? ctas : fit)), block(32 * kUpWarps);
    if (a.split > 1) {
        const cudaError_t e = allow_all_shared<ep_few_up_kernel<FROM, NT, true>>();
        return e != cudaSuccess ? e : launch_dependent(ep_few_up_kernel<FROM, NT, true>, grid, block, shared, s, a);
    }
    const cudaError_t e = allow_all_shared<ep_few_up_kernel<FROM, NT, false>>();
    return e != cudaSuccess ? e : launch_dependent(ep_few_up_kernel<FROM, NT, false>, grid, block, shared, s, a);
}

template <int NT>
cudaError_t launch_few(FewArgs a, int from, int sms, cudaStream_t s)
{
    // Warps to a unit: such that the last round of units, of the experts that rows name at most, leaves few warps idle; each
    // doubling costs some 5 %.
    const int64_t units = (int64_t)(a.pairs < a.experts ? a.pairs : a.experts) * (a.I / 16), at_once = (int64_t)sms * kUpWarpsPerSm<NT>;
    auto cost = [&](int split) {   // in units of one warp, times 1.05 per doubling
        return (double)((units * split + at_once - 1) / at_once) / split * (split == 1 ? 1.0 : split == 2 ? 1.05 : 1.1);
    };
    a.split = 1;
    for (int split = 2; split <= kUpWarps; split *= 2)
        if (cost(split) < cost(a.split)) a.split = split;
    cudaError_t e = from == kFromE4m3 ? launch_up<kFromE4m3, NT>(a, sms, s)
                    : from == kFromFp16 ? launch_up<kFromFp16, NT>(a, sms, s) : launch_up<kFromBf16, NT>(a, sms, s);
    if (e != cudaSuccess) return e;
    e = allow_all_shared<ep_few_down_kernel<NT>>();
    if (e != cudaSuccess) return e;
    // as many warps to a CTA as let all CTAs run at once; fewer where rows' sums would leave no room for the weights
    const int ctas = a.H / 16, per_sm = (ctas + sms - 1) / sms;
    int warps = per_sm < kDownWarpsPerSm<NT> ? kDownWarpsPerSm<NT> / per_sm : 1;
    auto shared = [&] {
        return entries_bytes(a.pairs, a.experts, a.rows) + (size_t)(a.pairs + 3) / 4 * 16 + (size_t)warps * a.rows * 64 +
               (size_t)warps * kDownAhead * kStepBytes;
    };
    while (shared() > 226 * 1024) --warps;   // ends: one warp of 4096 pairs and 1024 experts takes 84 KB
    return launch_dependent(ep_few_down_kernel<NT>, dim3(ctas), dim3(32 * warps), shared(), s, a);
}

size_t few_z_bytes(int64_t pairs, int inner) { return ((size_t)pairs * inner * 2 + 255) / 256 * 256; }

}  // namespace
}  // namespace ep

extern "C" size_t ep_moe_few_workspace_bytes(int64_t rows, int topk, int inner)
{
    using namespace ep;
    if (rows <= 0 || rows > kFewRows || topk < 1 || rows * topk > kFewPairs || inner < 16 || inner % 16 != 0 || inner > 1 << 19 ||
        rows * topk * inner >= (int64_t)1 << 31)
        return 0;
    return few_z_bytes(rows * topk, inner) + (size_t)rows * topk * (inner / 8);
}

extern "C" int ep_moe_few_rows(const void* x, const float* x_scales, int x_dtype, const int32_t* indices,
                               const float* weights, int64_t rows, int topk, int first_expert, int experts, int hidden,
                               int inner, const void* up, const float* up_scales, const void* down,
                               const float* down_scales, int out_dtype, void* out, void* workspace,
                               size_t workspace_bytes, void* stream)
{
    using namespace ep;
    const char* who = "ep_moe_few_rows";
    if (rows < 0 || rows > kFewRows)
        return layer_fail(EP_ERR_ARG, "%s: rows=%lld outside 0..%d: more rows are sorted by expert", who, (long long)rows, kFewRows);
    if (topk < 1 || rows * topk > kFewPairs)
        return layer_fail(EP_ERR_ARG, "%s: topk=%d is below 1, or rows*topk passes %d", who, topk, kFewPairs);
    if (experts < 1 || experts > kFewExperts)
        return layer_fail(EP_ERR_ARG, "%s: experts=%d outside 1..%d", who, experts, kFewExperts);
    if (hidden < 16 || hidden % 16 != 0 || hidden > 1 << 20)
        return layer_fail(EP_ERR_ARG, "%s: hidden=%d is not a multiple of 16 in 16..2^20", who, hidden);
    if (inner < 16 || inner % 16 != 0 || inner > 1 << 19)
        return layer_fail(EP_ERR_ARG, "%s: inner=%d is not a multiple of 16 in 16..2^19", who, inner);
    if (rows * topk * inner >= (int64_t)1 << 31)   // bytes of z are counted in 32 bits
        return layer_fail(EP_ERR_ARG, "%s: rows*topk*inner=%lld reaches 2^31", who, (long long)(rows * topk * inner));
    if (x_dtype != EP_FP8_E4M3 && x_dtype != EP_FP16 && x_dtype != EP_BF16)
        return layer_fail(EP_ERR_ARG, "%s: x_dtype=%d is not EP_FP8_E4M3, EP_FP16 or EP_BF16", who, x_dtype);
    if (out_dtype != EP_BF16 && out_dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "%s: out_dtype=%d is neither EP_BF16 nor EP_FP16", who, out_dtype);
    if (rows == 0) return EP_OK;
    if (!layer_aligned(x, 16) || (x_dtype == EP_FP8_E4M3) != (x_scales != nullptr) || (x_scales && !layer_aligned(x_scales, 4)))
        return layer_fail(EP_ERR_ARG, "%s: x is NULL or not 16-byte aligned, or x_scales is not given with e4m3 rows alone", who);
    if (!layer_aligned(indices, 4) || !layer_aligned(weights, 4))
        return layer_fail(EP_ERR_ARG, "%s: indices or weights is NULL or misaligned", who);
    if (!layer_aligned(up, 16) || !layer_aligned(down, 16) || !layer_aligned(up_scales, 4) || !layer_aligned(down_scales, 4))
        return layer_fail(EP_ERR_ARG, "%s: up, down or a scale array is NULL or misaligned", who);
    if (!layer_aligned(out, 16)) return layer_fail(EP_ERR_ARG, "%s: out is NULL or not 16-byte aligned", who);
    const size_t need = ep_moe_few_workspace_bytes(rows, topk, inner);
    if (!layer_aligned(workspace, 16) || workspace_bytes < need)
        return layer_fail(EP_ERR_ARG, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", who, workspace_bytes, need);
    FewArgs a{};
    a.x = (const uint8_t*)x; a.x_scales = x_scales; a.indices = indices; a.weights = weights;
    a.up = (const uint8_t*)up; a.up_scales = up_scales; a.down = (const uint8_t*)down; a.down_scales = down_scales;
    a.rows = (int)rows; a.k = topk; a.pairs = (int)rows * topk; a.first = first_expert; a.experts = experts;
    a.H = hidden; a.I = inner; a.hb = (hidden + 127) / 128; a.ib = (inner + 127) / 128; a.ub = (2 * inner + 127) / 128;
    a.z = (uint8_t*)workspace; a.z_exp = a.z + few_z_bytes(a.pairs, inner);
    a.out = out; a.out_fp16 = out_dtype == EP_FP16;
    const int sms = layer_num_sms();
    if (sms == 0) return layer_fail(EP_ERR_CUDA, "%s: cannot tell the current device's multiprocessors", who);
    const int from = x_dtype == EP_FP8_E4M3 ? kFromE4m3 : x_dtype == EP_FP16 ? kFromFp16 : kFromBf16;
    cudaStream_t s = (cudaStream_t)stream;
    // An expert's rows, at most all of them, in entries of 8 or 16.  Entries of 32 took longer even for 63 rows to each of 8
    // experts (221 against 212 us), because the sums leave fewer registers for warps.
    const cudaError_t e = rows <= 8 ? launch_few<1>(a, from, sms, s) : launch_few<2>(a, from, sms, s);
    return layer_cuda(e, "ep_moe_few_rows: launch");
}
