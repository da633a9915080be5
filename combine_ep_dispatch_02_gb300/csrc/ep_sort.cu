// ep_sort.cu -- rows sorted by expert, their weighted return, and the gradients of both.
//
// A pair is (row, top-k slot); its group is the global expert id in that slot if the expert lives
// on the row's rank.  The sort is stable: groups ascend, and within a group pairs keep their
// (row, slot) order, so results do not depend on the launch.
//   offsets[g]  sorted rows below group g            pos[pair]  the pair's sorted row, or -1
//   src[i]      the pair of sorted row i, -1 past offsets[groups]
//
// Sorting indices takes one CTA up to kSortSmallPairs pairs.  Above that, tiles of 2048 pairs are counted
// in one launch and placed in a second, whose CTAs each add up the counts of the tiles; above 64 tiles,
// tiles of 8192 pairs, and one CTA scans the counts (groups x tiles) in a launch between the two.
// 64 x 8 pairs and 256 groups take 2.5 us, 65536 pairs 8.2 us: two launches and a few trips to L2; 2 million
// pairs 44 us (56 with a dispatch's counts), mostly the one CTA's scan.
// Within a warp, __match_any_sync gives a pair's rank among equal groups; a warp's running counts
// live in shared memory, so no step has an order that atomics could change.
#include "ep_layer.cuh"

namespace ep {
namespace {

constexpr int kSortMaxGroups = 4096;
constexpr int kSortTileThreads = 256;
constexpr int kSortSteps = 8, kSortLongSteps = 32;   // steps of 256 pairs of a tile
constexpr int kSortShortTiles = 64;          // tiles of kSortSteps, at most; more pairs make longer tiles
constexpr int kSortSmallThreads = 512;       // one CTA for the whole sort
constexpr int kSortSmallSteps = 4;           // a step is 0.7 us in one CTA; the two launches take 6 to 9 us
constexpr int kSortSmallPairs = kSortSmallThreads * kSortSmallSteps;
constexpr int kSortSmallGroups = 2048;       // 16 warps' counts in 128 KB of shared memory

struct SortArgs {
    const int32_t* idx;
    const int32_t* counts;     // rows held by each rank, or NULL for all of them
    int32_t* offsets;
    int32_t* pos;
    int32_t* src;
    int32_t* tile_counts;      // [tiles][groups]
    int* status;
    int64_t pairs, max_rows;
    int64_t pairs_per_rank;
    int k, E, groups, tiles;
};

// Group of a pair, or -1.  Pairs of rows the rank did not receive are not read.
__device__ __forceinline__ int pair_group(const SortArgs& a, int64_t p)
{
    if (p >= a.pairs) return -1;
    int r = 0;
    if (a.pairs_per_rank != a.pairs) r = (int)((uint32_t)p / (uint32_t)a.pairs_per_rank);   // pairs < 2^31
    if (a.counts) {
        const int64_t in = p - r * a.pairs_per_rank;
        if (in >= (int64_t)a.counts[r] * a.k) return -1;
    }
    const int e = a.idx[p];
    return e >= r * a.E && e < (r + 1) * a.E ? e : -1;
}

// Rank of this lane's pair among the warp's earlier pairs of its group; count[] is the warp's.
__device__ __forceinline__ int warp_rank(int g, int* count, int lane)
{
    const unsigned same = __match_any_sync(0xffffffffu, g);
    int before = 0;
    if (g >= 0) before = count[g];
    __syncwarp();
    const unsigned lower = same & lanemask_lt();
    if (g >= 0 && lower == 0) count[g] = before + __popc(same);
    __syncwarp();
    return before + __popc(lower);
}

__device__ __forceinline__ void place_pair(const SortArgs& a, int64_t p, int g, int at)
{
    if (p >= a.pairs) return;
    if (g >= 0 && at >= a.max_rows) {
        record_status(a.status, EP_ERR_CAPACITY);
        g = -1;
    }
    a.pos[p] = g >= 0 ? at : -1;
    if (g >= 0) a.src[at] = (int32_t)p;
}

// Exclusive scan of one value per thread over the CTA; warp_sums holds one word per warp.
__device__ __forceinline__ int cta_exclusive_scan(int v, int* warp_sums, int& total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) warp_sums[w] = s;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < warps; ++i) {
        const int u = warp_sums[i];
        before += i < w ? u : 0;
        total += u;
    }
    return before + s - v;
}

__device__ __forceinline__ int clamp_rows(const SortArgs& a, int v) { return (int64_t)v < a.max_rows ? v : (int)a.max_rows; }

__global__ void __launch_bounds__(kSortSmallThreads) ep_sort_small_kernel(const SortArgs a)
{
    extern __shared__ int counts[];   // [warps][groups]
    __shared__ int warp_sums[32];
    constexpr int kWarps = kSortSmallThreads / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kWarps * a.groups; i += blockDim.x) counts[i] = 0;
    follow_predecessor();
    __syncthreads();
    const int steps = (int)((a.pairs + kSortSmallThreads - 1) / kSortSmallThreads);
    const int64_t first = (int64_t)w * steps * 32;   // a warp's pairs are consecutive
    int g[kSortSmallSteps], at[kSortSmallSteps];
#pragma unroll
    for (int i = 0; i < kSortSmallSteps; ++i) g[i] = i < steps ? pair_group(a, first + 32 * i + lane) : -1;
#pragma unroll
    for (int i = 0; i < kSortSmallSteps; ++i)
        if (i < steps) at[i] = warp_rank(g[i], counts + w * a.groups, lane);
    __syncthreads();
    int carry = 0;
    for (int b = 0; b < a.groups; b += blockDim.x) {
        const int e = b + threadIdx.x;
        int n = 0;
        if (e < a.groups)
            for (int v = 0; v < kWarps; ++v) n += counts[v * a.groups + e];
        int total;
        int base = carry + cta_exclusive_scan(n, warp_sums, total);
        if (e < a.groups) {
            a.offsets[e] = clamp_rows(a, base);
            for (int v = 0; v < kWarps; ++v) {
                const int c = counts[v * a.groups + e];
                counts[v * a.groups + e] = base;
                base += c;
            }
        }
        carry += total;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.offsets[a.groups] = clamp_rows(a, carry);
#pragma unroll
    for (int i = 0; i < kSortSmallSteps; ++i)
        if (i < steps) place_pair(a, first + 32 * i + lane, g[i], g[i] >= 0 ? counts[w * a.groups + g[i]] + at[i] : -1);
    for (int64_t i = carry + threadIdx.x; i < a.max_rows; i += blockDim.x) a.src[i] = -1;
}

__global__ void __launch_bounds__(kSortTileThreads) ep_sort_count_kernel(const SortArgs a, int tile_pairs)
{
    extern __shared__ int counts[];   // [groups]
    for (int i = threadIdx.x; i < a.groups; i += blockDim.x) counts[i] = 0;
    follow_predecessor();
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * tile_pairs;
#pragma unroll 8
    for (int i = threadIdx.x; i < tile_pairs; i += kSortTileThreads) {
        const int g = pair_group(a, first + i);
        if (g >= 0) atomicAdd(&counts[g], 1);   // whole numbers: the order does not matter
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.groups; i += blockDim.x)
        a.tile_counts[(int64_t)blockIdx.x * a.groups + i] = counts[i];
}

// Counts to first positions: tile_counts[t][g] becomes the sorted row of tile t's first pair of g.
// Groups are taken blockDim.x / kScanParts at a time, each column of tiles by kScanParts threads.
constexpr int kScanThreads = 1024, kScanParts = 8;
__global__ void __launch_bounds__(kScanThreads) ep_sort_scan_kernel(const SortArgs a)
{
    constexpr int kCols = kScanThreads / kScanParts;
    __shared__ int sums[kScanParts][kCols], warp_sums[32];
    follow_predecessor();
    const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
    const int per = (a.tiles + kScanParts - 1) / kScanParts;
    const int t0 = min(part * per, a.tiles), t1 = min(t0 + per, a.tiles);
    int carry = 0;
    for (int b = 0; b < a.groups; b += kCols) {
        const int g = b + col;
        int32_t* c = a.tile_counts + g;
        int n = 0;
        if (g < a.groups) {
#pragma unroll 8
            for (int t = t0; t < t1; ++t) n += c[(int64_t)t * a.groups];
        }
        sums[part][col] = n;
        __syncthreads();
        int all = 0, before = 0;
        for (int q = 0; q < kScanParts; ++q) {
            const int v = sums[q][col];
            before += q < part ? v : 0;
            all += v;
        }
        int total;
        int base = cta_exclusive_scan(part == 0 ? all : 0, warp_sums, total);
        __syncthreads();
        if (part == 0) sums[0][col] = base;   // threads of part 0 come first, in column order
        __syncthreads();
        base = carry + sums[0][col];
        if (g < a.groups) {
            if (part == 0) a.offsets[g] = clamp_rows(a, base);
            base += before;
#pragma unroll 8
            for (int t = t0; t < t1; ++t) {
                const int v = c[(int64_t)t * a.groups];
                c[(int64_t)t * a.groups] = base;
                base += v;
            }
        }
        carry += total;
        __syncthreads();
    }
    if (threadIdx.x == 0) a.offsets[a.groups] = clamp_rows(a, carry);
}

// SCANNED: tile_counts holds first positions and offsets is written; else tile_counts holds counts, and each
// CTA adds them up for itself.  The indices, too, are read after the wait, although the kernel before this one
// has waited for whoever wrote them: what another kernel wrote is visible to this one only after its own wait,
// and the count may have left their lines in L1.  Ranking them during that kernel would take 1.5 us less of 8.
template <int kSteps, bool SCANNED>
__global__ void __launch_bounds__(kSortTileThreads) ep_sort_place_kernel(const SortArgs a)
{
    extern __shared__ int counts[];   // [warps][groups]
    __shared__ int warp_sums[32];
    constexpr int kWarps = kSortTileThreads / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kWarps * a.groups; i += blockDim.x) counts[i] = 0;
    follow_predecessor();
    __syncthreads();
    const int64_t first = ((int64_t)blockIdx.x * kWarps + w) * kSteps * 32;
    int g[kSteps], at[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) g[i] = pair_group(a, first + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) at[i] = warp_rank(g[i], counts + w * a.groups, lane);
    __syncthreads();
    int carry = 0;
    for (int e0 = 0; e0 < a.groups; e0 += kSortTileThreads) {
        const int e = e0 + threadIdx.x;
        int base = 0;
        if constexpr (SCANNED) {
            if (e < a.groups) base = a.tile_counts[(int64_t)blockIdx.x * a.groups + e];
        } else {
            int all = 0, before = 0;
            if (e < a.groups) {
#pragma unroll 16
                for (int t = 0; t < a.tiles; ++t) {
                    const int c = a.tile_counts[(int64_t)t * a.groups + e];
                    all += c;
                    before += t < (int)blockIdx.x ? c : 0;
                }
            }
            int total;
            base = carry + cta_exclusive_scan(all, warp_sums, total);
            if (blockIdx.x == 0 && e < a.groups) a.offsets[e] = clamp_rows(a, base);
            base += before;
            carry += total;
        }
        if (e < a.groups)
            for (int v = 0; v < kWarps; ++v) {
                const int c = counts[v * a.groups + e];
                counts[v * a.groups + e] = base;
                base += c;
            }
    }
    if constexpr (SCANNED) carry = a.offsets[a.groups];
    else if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.groups] = clamp_rows(a, carry);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        place_pair(a, first + 32 * i + lane, g[i], g[i] >= 0 ? counts[w * a.groups + g[i]] + at[i] : -1);
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = carry + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < a.max_rows; i += step) a.src[i] = -1;
}

// ---------------------------------------------------------------- rows to expert order and back

struct RowsArgs {
    const uint8_t* in;        // x (sort) or y (return)
    const float* in_scales;
    const float* weights;     // [rows][k] or NULL (1)
    const int32_t* pos;
    const int32_t* counts;
    uint8_t* out;
    float* out_scales;
    const uint8_t* dout;      // return's gradient
    uint8_t* dy;
    float* dw;
    int* status;
    int64_t rows, rows_per_rank, max_rows;
    int64_t row_bytes;
    int k, sd, vecs;          // vecs: 16-byte vectors of a row
    int slices, slice_vecs;   // warps a row is split over, vectors each takes
};

__device__ __forceinline__ bool row_present(const RowsArgs& a, int64_t row)
{
    if (row >= a.rows) return false;
    if (!a.counts) return true;
    const int64_t r = a.rows_per_rank == a.rows ? 0 : row / a.rows_per_rank;
    return row - r * a.rows_per_rank < a.counts[r];
}

// A pair's sorted row, -1 if it has none; a row outside the buffer is recorded and skipped.
__device__ __forceinline__ int64_t checked_pos(const RowsArgs& a, int64_t pair)
{
    const int v = a.pos[pair];
    if (v >= 0 && v < a.max_rows) return v;
    if (v != -1) record_status(a.status, EP_ERR_DEVICE_BOUNDS);
    return -1;
}

constexpr int kRowThreads = 256;
constexpr int kWarpRowVecs = 128;   // a row's gradient is one warp's up to this many vectors
constexpr int kRowVecs = 4;   // vectors of a lane's slice at most: 2 KB of a row to a warp

// x rows to their sorted rows: each row is read once and written to each of its pairs.  HBM-bound by its
// stores: 8192 rows of 7168 BF16 to 65536 take 157 us, 6.7 TB/s.
__global__ void __launch_bounds__(kRowThreads) ep_sorted_rows_kernel(const RowsArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = unit / a.slices;
    const int slice = (int)(unit - row * a.slices);
    follow_predecessor();
    if (!row_present(a, row)) return;
    const uint8_t* x = a.in + row * a.row_bytes;
    uint4 v[kRowVecs];
    const int v0 = slice * a.slice_vecs + lane, v1 = min(a.vecs, (slice + 1) * a.slice_vecs);
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i)
        if (v0 + 32 * i < v1) v[i] = ld_stream_v4(x + 16 * (int64_t)(v0 + 32 * i));
    for (int jb = 0; jb < a.k; jb += 32) {
        const int64_t mine = jb + lane < a.k ? checked_pos(a, row * a.k + jb + lane) : -1;
        for (int j = 0; j < min(32, a.k - jb); ++j) {
            const int64_t to = __shfl_sync(0xffffffffu, mine, j);
            if (to < 0) continue;
            uint8_t* out = a.out + to * a.row_bytes;
#pragma unroll
            for (int i = 0; i < kRowVecs; ++i)
                if (v0 + 32 * i < v1) st_v4(out + 16 * (int64_t)(v0 + 32 * i), v[i]);
            if (slice == 0)
                for (int i = lane; i < a.sd; i += 32) a.out_scales[to * a.sd + i] = a.in_scales[row * a.sd + i];
        }
    }
}

// out[row] = round(sum over slots, ascending, of weight * y[pos]); FP32 sums.  A warp takes a.slice_vecs
// vectors of a row.  Reading HBM at full rate takes about 100 KB on their way to each SM: a lane loads
// the next vector of up to kSlots rows before it adds the current ones, so 16 warps keep up to 128 KB
// in flight without a gap: 8192 rows of 7168 BF16 from 65536, 164 us, 6.4 TB/s (192 us without).
template <bool FP16, int kSlots>
__global__ void __launch_bounds__(kRowThreads, 2) ep_return_rows_kernel(const RowsArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = unit / a.slices;
    const int slice = (int)(unit - row * a.slices);
    follow_predecessor();
    if (!row_present(a, row)) return;
    int mine = -1;
    float weight = 0.0f;
    if (lane < a.k) {
        mine = (int)checked_pos(a, row * a.k + lane);
        if (mine >= 0) weight = a.weights ? a.weights[row * a.k + lane] : 1.0f;
    }
    int from[kSlots];
    float w[kSlots];
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
        from[j] = __shfl_sync(0xffffffffu, mine, j);
        w[j] = __shfl_sync(0xffffffffu, weight, j);
    }
    const int v0 = slice * a.slice_vecs, v1 = min(a.vecs, v0 + a.slice_vecs);
    auto load = [&](uint4 (&y)[kSlots], int v) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            y[j] = make_uint4(0, 0, 0, 0);
            if (from[j] >= 0 && v < v1) y[j] = ld_stream_v4(a.in + from[j] * a.row_bytes + 16 * (int64_t)v);
        }
    };
    auto fold = [&](const uint4 (&y)[kSlots], int v) {
        float acc[8] = {};
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            float f[8];
            unpack8<FP16>(y[j], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[j], f[q], acc[q]);
        }
        if (v < v1) st_v4(a.out + row * a.row_bytes + 16 * (int64_t)v, pack8<FP16>(acc));
    };
    uint4 y0[kSlots], y1[kSlots];
    int v = v0 + lane;
    load(y0, v);
    for (; v - lane < v1; v += 64) {
        load(y1, v + 32);
        fold(y0, v);
        load(y0, v + 64);
        fold(y1, v + 32);
    }
}

// The same for more than 8 slots a row, 8 at a time.
template <bool FP16>
__global__ void __launch_bounds__(kRowThreads) ep_return_rows_many_kernel(const RowsArgs a)
{
    constexpr int kSlots = 8;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = unit / a.slices;
    const int slice = (int)(unit - row * a.slices);
    follow_predecessor();
    if (!row_present(a, row)) return;
    const int v0 = slice * a.slice_vecs, v1 = min(a.vecs, v0 + a.slice_vecs);
    int64_t from[2] = {-1, -1};   // of slots lane and lane + 32
    float weight[2] = {0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (32 * h + lane < a.k) {
            from[h] = checked_pos(a, row * a.k + 32 * h + lane);
            if (from[h] >= 0) weight[h] = a.weights ? a.weights[row * a.k + 32 * h + lane] : 1.0f;
        }
    for (int v = v0 + lane; v - lane < v1; v += 32) {
        float acc[8] = {};
        for (int jb = 0; jb < a.k; jb += kSlots) {
            uint4 y[kSlots];
            float w[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                const int64_t r = __shfl_sync(0xffffffffu, jb < 32 ? from[0] : from[1], (jb + j) & 31);
                w[j] = __shfl_sync(0xffffffffu, jb < 32 ? weight[0] : weight[1], (jb + j) & 31);
                y[j] = make_uint4(0, 0, 0, 0);
                if (r >= 0 && v < v1) y[j] = ld_stream_v4(a.in + r * a.row_bytes + 16 * (int64_t)v);
            }
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                float f[8];
                unpack8<FP16>(y[j], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[j], f[q], acc[q]);
            }
        }
        if (v < v1) st_v4(a.out + row * a.row_bytes + 16 * (int64_t)v, pack8<FP16>(acc));
    }
}

// Gradient of the weighted return: dy[pos] = round(weight * dout[row]), dw = <y[pos], dout[row]>.  A row
// is one warp's, or one CTA's, so that each dot product is summed in one place and in one order; the
// products of kSlots slots run together.  HBM-bound: 4096 rows of 7168 BF16 and 8 slots 151 us, 6.6 TB/s.
template <bool FP16, bool WARP, int kSlots>
__global__ void __launch_bounds__(kRowThreads) ep_return_rows_backward_kernel(const RowsArgs a)
{
    __shared__ float part[kRowThreads / 32][kSlots];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = WARP ? (int64_t)blockIdx.x * (kRowThreads / 32) + warp : blockIdx.x;
    follow_predecessor();
    if (!row_present(a, row)) return;   // whole warps, and whole CTAs where they synchronise
    const uint8_t* dout = a.dout + row * a.row_bytes;
    for (int jb = 0; jb < a.k; jb += kSlots) {
        int at[kSlots];
        float wt[kSlots], dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            at[j] = jb + j < a.k ? (int)checked_pos(a, row * a.k + jb + j) : -1;
            wt[j] = at[j] >= 0 ? a.weights[row * a.k + jb + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int v = WARP ? lane : threadIdx.x; v < a.vecs; v += WARP ? 32 : kRowThreads) {
            uint4 y[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (at[j] >= 0) y[j] = ld_stream_v4(a.in + at[j] * a.row_bytes + 16 * (int64_t)v);
            float g[8];
            unpack8<FP16>(*reinterpret_cast<const uint4*>(dout + 16 * (int64_t)v), g);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (at[j] < 0) continue;
                float f[8], o[8];
                unpack8<FP16>(y[j], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    dot[j] = fmaf(f[q], g[q], dot[j]);
                    o[q] = wt[j] * g[q];
                }
                st_v4(a.dy + at[j] * a.row_bytes + 16 * (int64_t)v, pack8<FP16>(o));
            }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if (lane == j) part[warp][j] = dot[j];
        }
        if constexpr (WARP) {
            __syncwarp();
            if (lane < kSlots && jb + lane < a.k) a.dw[row * a.k + jb + lane] = part[warp][lane];
            __syncwarp();
        } else {
            __syncthreads();
            if (threadIdx.x < kSlots && jb + (int)threadIdx.x < a.k) {
                float s = 0.0f;
                for (int i = 0; i < kRowThreads / 32; ++i) s += part[i][threadIdx.x];
                a.dw[row * a.k + jb + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

template <bool FP16>
cudaError_t launch_return(const RowsArgs& a, unsigned grid, cudaStream_t s)
{
    auto* kernel = a.k <= 2   ? ep_return_rows_kernel<FP16, 2>
                   : a.k <= 4 ? ep_return_rows_kernel<FP16, 4>
                   : a.k <= 8 ? ep_return_rows_kernel<FP16, 8>
                              : ep_return_rows_many_kernel<FP16>;
    return launch_dependent(kernel, dim3(grid), dim3(kRowThreads), 0, s, a);
}

template <bool FP16>
cudaError_t launch_return_backward(const RowsArgs& a, cudaStream_t s)
{
    const bool warp = a.vecs <= kWarpRowVecs;
    const unsigned grid = (unsigned)(warp ? (a.rows + kRowThreads / 32 - 1) / (kRowThreads / 32) : a.rows);
    // 8 slots together shorten one row's chain of loads; with every SM full their registers cost more.  us, 4 slots
    // against 8, rows of 8 slots: of 7168, 64 rows 9.3 : 6.9, 256 11.3 : 9.9, 512 17.4 : 18.4, 768 33.9 : 33.5,
    // 1024 42.9 : 44.5, 4096 151.5 : 157.0; of 2048, 256 rows 5.1 : 4.7, 512 7.3 : 7.8, 1024 11.1 : 12.8, 4096
    // 45.8 : 55.0.  Between 512 and 1024 rows neither is ahead at every width; the bound suits the widest.
    auto* kernel = warp ? (a.k <= 4 ? ep_return_rows_backward_kernel<FP16, true, 4>
                                    : ep_return_rows_backward_kernel<FP16, true, 8>)
                        : (a.k <= 4 || a.rows >= 1024 ? ep_return_rows_backward_kernel<FP16, false, 4>
                                                      : ep_return_rows_backward_kernel<FP16, false, 8>);
    return launch_dependent(kernel, dim3(grid), dim3(kRowThreads), 0, s, a);
}

// The shape every call of this file shares.
int check_rows(const char* who, int W, int64_t rows_per_rank, int k, int64_t max_rows, const int32_t* counts,
               const int32_t* device_status)
{
    if (W < 1 || W > kMaxRanks) return layer_fail(EP_ERR_ARG, "%s: W=%d outside 1..%d", who, W, kMaxRanks);
    if (k < 1 || k > kMaxTopk) return layer_fail(EP_ERR_ARG, "%s: topk=%d outside 1..%d", who, k, kMaxTopk);
    if (rows_per_rank < 0 || (int64_t)W * k * rows_per_rank >= (int64_t)1 << 31 || rows_per_rank >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: W*rows_per_rank*topk=%d*%lld*%d outside 0..2^31-1", who, W,
                          (long long)rows_per_rank, k);
    if (max_rows < 0 || max_rows >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: max_rows=%lld outside 0..2^31-1", who, (long long)max_rows);
    if (counts && !layer_aligned(counts, 4)) return layer_fail(EP_ERR_ARG, "%s: counts is not 4-byte aligned", who);
    if (!layer_aligned(device_status, 4))
        return layer_fail(EP_ERR_ARG, "%s: device_status is NULL or not 4-byte aligned", who);
    return EP_OK;
}

int check_row_type(const char* who, int dtype, int hidden)
{
    if (dtype != EP_BF16 && dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "%s: dtype=%d is neither EP_BF16 nor EP_FP16", who, dtype);
    if (hidden < 8 || hidden % 8 != 0 || hidden >= 1 << 30)
        return layer_fail(EP_ERR_ARG, "%s: hidden=%d is not a positive multiple of 8 below 2^30", who, hidden);
    return EP_OK;
}

int sort_tile_pairs(int64_t pairs)
{
    return kSortTileThreads * (pairs <= (int64_t)kSortShortTiles * kSortTileThreads * kSortSteps ? kSortSteps : kSortLongSteps);
}

// One at least: no pairs in more groups than one CTA counts still leave offsets and src to write.
int64_t sort_tiles(int64_t pairs)
{
    return pairs == 0 ? 1 : (pairs + sort_tile_pairs(pairs) - 1) / sort_tile_pairs(pairs);
}

bool sort_is_small(int64_t pairs, int groups) { return pairs <= kSortSmallPairs && groups <= kSortSmallGroups; }

// Splits rows into slices of about equal length, at most `most` steps of 32 vectors, and gives the CTAs of 8
// warps that take one each.  Of the splits, the one with the fewest waves of resident warps times steps,
// where a slice's start (positions, first loads) counts as a step and a half: 300 rows of 8 x 7168 return in
// 8 slices, one wave, 7.6 us, in 14 slices, two waves, 8.6 us.
int set_slices(const char* who, RowsArgs& a, int most, int warps_per_sm, unsigned& grid)
{
    a.vecs = (int)(a.row_bytes / 16);
    const int64_t steps = (a.vecs + 31) / 32, least = (steps + most - 1) / most;
    const int64_t ctas = (a.rows * least + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (ctas >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: %lld rows of %lld bytes need %lld CTAs, past 2^31-1", who, (long long)a.rows,
                          (long long)a.row_bytes, (long long)ctas);
    const int64_t resident = (int64_t)warps_per_sm * layer_num_sms();
    if (resident == 0) return layer_fail(EP_ERR_CUDA, "%s: cannot tell the current device's multiprocessors", who);
    int64_t best = -1;
    for (int64_t n = least; n <= steps && n < least + 64; ++n) {
        const int64_t cost = (a.rows * n + resident - 1) / resident * (2 * ((steps + n - 1) / n) + 3);
        if (best < 0 || cost < best) {
            best = cost;
            a.slices = (int)n;
        }
        if (a.rows * n >= 4 * resident) break;   // further splits only add starts
    }
    a.slice_vecs = (int)((steps + a.slices - 1) / a.slices) * 32;
    grid = (unsigned)((a.rows * a.slices + kRowThreads / 32 - 1) / (kRowThreads / 32));   // `ctas`, or under 2^20
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" {

size_t ep_sort_workspace_bytes(int W, int64_t rows_per_rank, int topk, int experts_per_rank)
{
    using namespace ep;
    if (W < 1 || W > kMaxRanks || rows_per_rank < 0 || rows_per_rank >= (int64_t)1 << 31 || topk < 1 ||
        topk > kMaxTopk || experts_per_rank < 1 || (int64_t)W * experts_per_rank > kSortMaxGroups)
        return 0;
    const int64_t pairs = (int64_t)W * rows_per_rank * topk;
    if (pairs >= (int64_t)1 << 31 || sort_is_small(pairs, W * experts_per_rank)) return 0;
    return (size_t)sort_tiles(pairs) * W * experts_per_rank * sizeof(int32_t);
}

int ep_sort_by_expert(const int32_t* indices, const int32_t* counts, int W, int64_t rows_per_rank, int topk,
                      int experts_per_rank, int64_t max_rows, int32_t* offsets, int32_t* pos, int32_t* src,
                      void* workspace, size_t workspace_bytes, int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_sort_by_expert";
    if (int rc = check_rows(who, W, rows_per_rank, topk, max_rows, counts, device_status)) return rc;
    if (experts_per_rank < 1 || (int64_t)W * experts_per_rank > kSortMaxGroups)
        return layer_fail(EP_ERR_ARG, "%s: W*experts_per_rank=%d*%d outside 1..%d", who, W, experts_per_rank,
                          kSortMaxGroups);
    SortArgs a{};
    a.pairs_per_rank = rows_per_rank * topk;
    a.pairs = W * a.pairs_per_rank;
    if (!layer_aligned(offsets, 4)) return layer_fail(EP_ERR_ARG, "%s: offsets is NULL or not 4-byte aligned", who);
    if (a.pairs > 0 && (!layer_aligned(indices, 4) || !layer_aligned(pos, 4)))
        return layer_fail(EP_ERR_ARG, "%s: indices or pos is NULL or not 4-byte aligned", who);
    if (max_rows > 0 && !layer_aligned(src, 4))
        return layer_fail(EP_ERR_ARG, "%s: src is NULL or not 4-byte aligned", who);
    const size_t need = ep_sort_workspace_bytes(W, rows_per_rank, topk, experts_per_rank);
    if (need > 0 && (!layer_aligned(workspace, 4) || workspace_bytes < need))
        return layer_fail(EP_ERR_ARG, "%s: the workspace is NULL, misaligned or holds %zu of %zu bytes", who,
                          workspace_bytes, need);
    a.idx = indices; a.counts = counts; a.offsets = offsets; a.pos = pos; a.src = src;
    a.tile_counts = (int32_t*)workspace; a.status = device_status;
    a.max_rows = max_rows; a.k = topk; a.E = experts_per_rank; a.groups = W * experts_per_rank;
    a.tiles = (int)sort_tiles(a.pairs);
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (sort_is_small(a.pairs, a.groups)) {
        const size_t smem = (size_t)(kSortSmallThreads / 32) * a.groups * sizeof(int);
        e = allow_all_shared<ep_sort_small_kernel>();
        if (e == cudaSuccess) e = launch_dependent(ep_sort_small_kernel, dim3(1), dim3(kSortSmallThreads), smem, s, a);
        return layer_cuda(e, "ep_sort_by_expert: launch");
    }
    const size_t smem = (size_t)(kSortTileThreads / 32) * a.groups * sizeof(int);
    const int tile_pairs = sort_tile_pairs(a.pairs);
    const bool shorter = tile_pairs == kSortTileThreads * kSortSteps;
    auto* place = shorter ? ep_sort_place_kernel<kSortSteps, false> : ep_sort_place_kernel<kSortLongSteps, true>;
    e = shorter ? allow_all_shared<ep_sort_place_kernel<kSortSteps, false>>()
                : allow_all_shared<ep_sort_place_kernel<kSortLongSteps, true>>();
    if (e == cudaSuccess)
        e = launch_dependent(ep_sort_count_kernel, dim3(a.tiles), dim3(kSortTileThreads), a.groups * sizeof(int), s, a,
                             tile_pairs);
    if (e == cudaSuccess && !shorter) e = launch_dependent(ep_sort_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, a);
    if (e == cudaSuccess) e = launch_dependent(place, dim3(a.tiles), dim3(kSortTileThreads), smem, s, a);
    return layer_cuda(e, "ep_sort_by_expert: launch");
}

int ep_sorted_rows(const void* x, const float* scales, const int32_t* pos, const int32_t* counts, int W,
                   int64_t rows_per_rank, int topk, int64_t max_rows, int64_t row_bytes, int scale_dim, void* out,
                   float* out_scales, int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_sorted_rows";
    if (int rc = check_rows(who, W, rows_per_rank, topk, max_rows, counts, device_status)) return rc;
    if (row_bytes < 16 || row_bytes % 16 != 0 || row_bytes >= (int64_t)1 << 31)
        return layer_fail(EP_ERR_ARG, "%s: a row of %lld bytes is not a positive multiple of 16 below 2^31", who,
                          (long long)row_bytes);
    if (scale_dim < 0 || scale_dim > 65536)
        return layer_fail(EP_ERR_ARG, "%s: scale_dim=%d outside 0..65536", who, scale_dim);
    if (rows_per_rank == 0 || max_rows == 0) return EP_OK;
    if (!layer_aligned(x, 16) || !layer_aligned(out, 16) || !layer_aligned(pos, 4))
        return layer_fail(EP_ERR_ARG, "%s: x, out or pos is NULL or misaligned", who);
    if (scale_dim > 0 && (!layer_aligned(scales, 4) || !layer_aligned(out_scales, 4)))
        return layer_fail(EP_ERR_ARG, "%s: scale_dim=%d needs scales and out_scales, 4-byte aligned", who, scale_dim);
    RowsArgs a{};
    a.in = (const uint8_t*)x; a.in_scales = scales; a.pos = pos; a.counts = counts; a.out = (uint8_t*)out;
    a.out_scales = out_scales; a.status = device_status; a.rows = W * rows_per_rank; a.rows_per_rank = rows_per_rank;
    a.max_rows = max_rows; a.row_bytes = row_bytes; a.k = topk; a.sd = scale_dim;
    unsigned grid;
    if (int rc = set_slices(who, a, kRowVecs, 40, grid)) return rc;
    return layer_cuda(launch_dependent(ep_sorted_rows_kernel, dim3(grid), dim3(kRowThreads), 0, (cudaStream_t)stream, a),
                      "ep_sorted_rows: launch");
}

int ep_return_rows(const void* y, const float* weights, const int32_t* pos, const int32_t* counts, int W,
                   int64_t rows_per_rank, int topk, int64_t max_rows, int hidden, int dtype, void* out,
                   int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_return_rows";
    if (int rc = check_rows(who, W, rows_per_rank, topk, max_rows, counts, device_status)) return rc;
    if (int rc = check_row_type(who, dtype, hidden)) return rc;
    if (rows_per_rank == 0) return EP_OK;
    if ((max_rows > 0 && !layer_aligned(y, 16)) || !layer_aligned(out, 16) || !layer_aligned(pos, 4))
        return layer_fail(EP_ERR_ARG, "%s: y, out or pos is NULL or misaligned", who);
    if (weights && !layer_aligned(weights, 4)) return layer_fail(EP_ERR_ARG, "%s: weights is not 4-byte aligned", who);
    RowsArgs a{};
    a.in = (const uint8_t*)y; a.weights = weights; a.pos = pos; a.counts = counts; a.out = (uint8_t*)out;
    a.status = device_status; a.rows = W * rows_per_rank; a.rows_per_rank = rows_per_rank; a.max_rows = max_rows;
    a.row_bytes = 2 * (int64_t)hidden; a.k = topk;
    unsigned grid;
    if (int rc = set_slices(who, a, 8, 16, grid)) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == EP_FP16 ? launch_return<true>(a, grid, s) : launch_return<false>(a, grid, s);
    return layer_cuda(e, "ep_return_rows: launch");
}

int ep_return_rows_backward(const void* y, const float* weights, const void* dout, const int32_t* pos,
                            const int32_t* counts, int W, int64_t rows_per_rank, int topk, int64_t max_rows,
                            int hidden, int dtype, void* dy, float* dweights, int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_return_rows_backward";
    if (int rc = check_rows(who, W, rows_per_rank, topk, max_rows, counts, device_status)) return rc;
    if (int rc = check_row_type(who, dtype, hidden)) return rc;
    if (rows_per_rank == 0) return EP_OK;
    if ((max_rows > 0 && (!layer_aligned(y, 16) || !layer_aligned(dy, 16))) || !layer_aligned(dout, 16) ||
        !layer_aligned(pos, 4))
        return layer_fail(EP_ERR_ARG, "%s: y, dout, dy or pos is NULL or misaligned", who);
    if (!layer_aligned(weights, 4) || !layer_aligned(dweights, 4))
        return layer_fail(EP_ERR_ARG, "%s: weights or dweights is NULL or not 4-byte aligned", who);
    RowsArgs a{};
    a.in = (const uint8_t*)y; a.weights = weights; a.pos = pos; a.counts = counts; a.dout = (const uint8_t*)dout;
    a.dy = (uint8_t*)dy; a.dw = dweights; a.status = device_status; a.rows = W * rows_per_rank;
    a.rows_per_rank = rows_per_rank; a.max_rows = max_rows; a.row_bytes = 2 * (int64_t)hidden; a.k = topk;
    a.vecs = hidden / 8;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == EP_FP16 ? launch_return_backward<true>(a, s) : launch_return_backward<false>(a, s);
    return layer_cuda(e, "ep_return_rows_backward: launch");
}

}  // extern "C"
