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
#include "ep_tcgen05.cuh"

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
    int columns, nb;          // rows of b in one group, and their 128-row blocks
    int swiglu, dtype;
    int vec;                  // rows take 32-byte (2) or 16-byte (1) stores, or neither
};

// First and last row of group g, clamped to the buffer; off is p.offsets or a copy of it.
__device__ __forceinline__ void group_rows(const MatmulArgs& p, const int32_t* off, int g, int& lo, int& hi)
{
    if (!off) { lo = 0; hi = (int)p.rows; return; }
    lo = max(0, min(off[g], (int)p.rows));
    hi = max(lo, min(off[g + 1], (int)p.rows));
}

// ---- tiles of 128 rows
//
// A CTA keeps one SM and walks output tiles of 128 rows by 256 rows of b (with SwiGLU: 128 gate rows and
// the 128 up rows that belong to them).  Warp 0 loads 128-byte wide K blocks of both operands by TMA
// into kStages shared-memory stages; warp 1 multiplies each block on the tensor cores into one of two
// 256-column accumulators in tensor memory; warps 2 and 3 multiply the block's row and column scales
// into a shared-memory ring; eight warps add each block's sums, times those factors, to FP32
// registers while the next block is multiplied.  The scales differ from block to block of K, so the
// sums cannot stay in tensor memory over a tile.
//
// What bounds it is not settled.  A block takes 690 cycles, of which its products need 512 (128*256*128 at 8192 a
// cycle; 528 measured alone).  An accumulator's way takes 1220 (multiplied in 512, 300 until the scaling warps are
// told and the multiplying warp is told back, 400 until they have read it), and tensor memory holds two: 610 a
// block.  But shortening that way did not help: two 128-column products a block, with two accumulators each, took
// 703 cycles (a is read twice).  Loading half of b's bytes takes a block to 664 cycles, none to 650.
// What it took to get there, of 1340 cycles at first: descriptors and loop counts in uniform registers; an
// accumulator given back over a named barrier, because a hop over an mbarrier takes 300 cycles; factors
// made ahead by idle warps; 32 columns read while the 32 before are added, across the ends of blocks.
// 256 columns, because a 128-column product takes 68 cycles where half of a 256-column one takes 64, and
// reads the rows again; where tiles are too few for the SMs, tiles of 128 columns, or a tile's K by
// several CTAs, are shorter.
//
// 32768 rows in 32 groups, 7168 x 4096 with SwiGLU: 690 to 706 us, 2790 TFLOP/s (0.73 of twice the measured BF16
// rate), and 805 to 840 us once the card holds its power limit, at 1545 MHz.  2048 x 7168: 400 us, whose 16 blocks
// a tile cannot hide the tile's end, 3000 cycles.

constexpr int kTileRows = 128, kTileCols = 256, kBlockK = 128;
constexpr int kStages = 4;             // even: a stage always goes to the same accumulator
__host__ __device__ constexpr int stage_bytes(int cols) { return (kTileRows + cols) * kBlockK; }
constexpr int kScaleWarps = 8;         // two to a quarter of the lanes, 128 columns each
constexpr int kScaleThreads = 32 * kScaleWarps;
constexpr int kProductThreads = 128 + kScaleThreads;   // load, multiply, two factor warps; the scaling warps
constexpr int kInfo = 16;              // more tiles than the loading warp can be ahead of the scaling warps: 8
constexpr int kChunkTiles = 16;        // row tiles that share b's columns before the next columns
constexpr int kFactors = 3;            // factors of a row and block: per half, or gate and two up blocks
constexpr int kRing = 8;               // blocks of factors: a block is written when the block kStages before it has
                                       // been multiplied, while up to kStages + 3 before it may be unread
constexpr int kRingFloats = kRing * kFactors * kTileRows;
constexpr int kSharedBlocks = 24;     // blocks of K from which CTAs may share a tile of 128 rows
constexpr int kMaxSplit = 8;          // CTAs that share a tile's K, at most: 1, 2, 4 or 8
constexpr int kSharedOffsets = 512;    // groups whose offsets are copied to shared memory

struct Tile {
    int g, m0, m1, n0;   // group, first row, end of the group's rows, first output column
};

// Exclusive prefix of the groups' tile counts, by one warp.
template <int ROWS>
__device__ __forceinline__ void scan_tiles(const MatmulArgs& p, int* first, int col_tiles, int lane)
{
    int carry = 0;
    for (int b = 0; b < p.groups; b += 32) {
        int n = 0;
        if (b + lane < p.groups) {
            int lo, hi;
            group_rows(p, p.offsets, b + lane, lo, hi);
            n = (hi - lo + ROWS - 1) / ROWS * col_tiles;
        }
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (b + lane < p.groups) first[b + lane] = carry + s - n;
        carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) first[p.groups] = carry;
}

// a / b for whole numbers, b > 0, without an integer division where a is small: (a + 0.5) / b is at least
// 0.5 / b away from a whole number, and below 2^21 the float quotient is off by less.
__device__ __forceinline__ int quick_div(int a, int b)
{
    if (a < 1 << 21) return (int)__fdividef((float)a + 0.5f, (float)b);
    return a / b;
}

// Tile t, by a converged warp: groups in order; within a group, chunks of kChunkTiles row tiles, whose rows and
// the group's weights stay in L2 while the chunk is done; within a chunk, row tiles before columns.
template <int ROWS, int COLS>
__device__ __forceinline__ Tile find_tile(const MatmulArgs& p, const int32_t* off, const int* first, int col_tiles,
                                          int t)
{
    // the last group whose first tile is not past t, 32 candidates at a time
    int lo = 0;
    for (int n = p.groups; n > 1;) {
        const int step = (n + 31) >> 5, at = lo + (int)(threadIdx.x & 31) * step;
        const unsigned m = __ballot_sync(0xffffffffu, at < lo + n && first[min(at, p.groups)] <= t);
        const int skip = (__popc(m) - 1) * step;
        lo += skip;
        n = min(step, n - skip);
    }
    Tile x;
    x.g = lo;
    int r0;
    group_rows(p, off, lo, r0, x.m1);
    const int tiles = (x.m1 - r0 + ROWS - 1) / ROWS;
    const int in = t - first[lo], wide_tiles = kChunkTiles * col_tiles;
    const int chunk = quick_div(in, wide_tiles), rest = in - chunk * wide_tiles;
    const int wide = min(kChunkTiles, tiles - chunk * kChunkTiles);
    const int col = quick_div(rest, wide);
    x.m0 = r0 + (chunk * kChunkTiles + rest - col * wide) * ROWS;
    x.n0 = col * COLS;
    return x;
}

// 32 accumulator columns times the factor, added to 32 of a thread's sums.
__device__ __forceinline__ void add_scaled(float2* acc, const uint32_t (&r)[32], float s)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        fma2(acc[i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), make_float2(s, s));
}

// The same where columns from `split` on, an even number, take another factor (an up block that ends
// inside the tile).
__device__ __forceinline__ void add_scaled(float2* acc, const uint32_t (&r)[32], float lo, float hi, int split)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s = 2 * i < split ? lo : hi;
        fma2(acc[i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), make_float2(s, s));
    }
}

// 2 * PAIRS consecutive columns, n of which exist, of a warp's 32 rows, m of which exist (row by lane, rows `pitch`
// bytes apart), 16-bit.  A store of 32 bytes by every lane to a row of its own visits 32 lines, two
// cycles each, 4000 for a tile.  So four lanes first trade 32-byte pieces, two exchanges of half of
// them, until lane q of the four holds piece q (then q + 4) of all four rows: a store then writes 128
// bytes each of 8 rows.
template <bool FP16, int PAIRS>
__device__ __forceinline__ void store_rows(uint8_t* out, int64_t pitch, const float2 (&acc)[PAIRS], int m, int n, int vec)
{
    const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
    for (int h = 0; h < PAIRS / 32; ++h) {
        uint32_t w[4][8];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = acc[32 * h + 8 * c + i];
                w[c][i] = pack2<FP16>(v.x, v.y);
            }
#pragma unroll
        for (int bit = 1; bit <= 2; bit *= 2) {
            const bool upper = q & bit;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c & bit) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? w[c][i] : w[c | bit][i], bit);
                    if (upper) w[c][i] = got;
                    else w[c | bit][i] = got;
                }
            }
        }
        const int left = n - (64 * h + 16 * q);   // columns of this lane's pieces that exist
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = (lane & ~3) + r;
            if (row >= m) break;
            uint8_t* to = out + row * pitch + 128 * h + 32 * q;
            if (vec == 2 && left >= 16) {
                st_v8(to, make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]), make_uint4(w[r][4], w[r][5], w[r][6], w[r][7]));
            } else if (vec == 1 && left >= 16) {
                st_v4(to, make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]));
                st_v4(to + 16, make_uint4(w[r][4], w[r][5], w[r][6], w[r][7]));
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < left) reinterpret_cast<uint16_t*>(to)[i] = (uint16_t)(w[r][i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

// gate * sigmoid(gate) * up, in this order: gate * up could pass FP32's range where the result is far inside.
// The exponential's argument is split, so that its rounding does not enter (the product with log2 e alone would
// be off by |gate| units in the exponential's last place).  What stays is that of log2 e to FP32, 1.9e-8 of the
// gate, and two units of each approximate instruction: in all 2 units at a gate of -10, 5 at -40, 11 at -87,
// which the e4m3 code's 2^-4 hides.  Below -88 the exponential is held at 2^127, whose reciprocal is 0: a sigmoid
// under FP32's smallest normal number counts as 0.  An infinite gate's split is not a number, which fminf turns
// into one that changes neither 0 nor 2^127's 0.
__device__ __forceinline__ float swiglu(float gate, float up)
{
    const float t = -1.4426950408889634f * gate;
    const float rest = fminf(fmaf(-1.4426950408889634f, gate, -t), 1.0f);   // what rounding t dropped
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fminf(t, 127.0f)));
    e = fmaf(e * 0.6931471805599453f, rest, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return gate * r * up;
}

// Named barriers 1 to 4, one to an accumulator: it has been read.  Every scaling warp arrives once per block,
// in every case; the multiplying warp waits before it writes that accumulator again.
constexpr int kReadThreads = kScaleThreads + 32;
__device__ __forceinline__ void read_arrive(uint32_t buf)
{
    asm volatile("bar.arrive %0, %1;" :: "r"(1 + buf), "n"(kReadThreads) : "memory");
}
__device__ __forceinline__ void read_wait(uint32_t buf)
{
    asm volatile("bar.sync %0, %1;" :: "r"(1 + buf), "n"(kReadThreads) : "memory");
}

// 4 consecutive 16-bit outputs at element `at`, `left` of which exist.
__device__ __forceinline__ void store4(const MatmulArgs& p, int64_t at, const float4& v, int left)
{
    uint2 w;
    if (p.dtype == EP_FP16) w = make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w));
    else w = make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
    uint16_t* out = (uint16_t*)p.out + at;
    if (p.vec >= 1 && left >= 4) {
        *reinterpret_cast<uint2*>(out) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) out[i] = (uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
    }
}

// A tile whose K the S CTAs of a cluster shared: this CTA finishes rows r .. r_end - 1 of those that are
// kScaleWarps apart, from every CTA's sums at address `sums`, added in the CTAs' order.  A lane takes 4
// columns and the 4 that are 128 further on; 16 loads are on their way before the first is added, from all
// CTAs alike, so that no CTA's shared memory is asked by all of them at once.
template <bool SWIGLU, int S>
__device__ __forceinline__ void finish_rows(const MatmulArgs& p, const Tile& x, uint32_t sums, int r, int r_end)
{
    constexpr int kRows = 8 / S;
    const int lane = threadIdx.x & 31;
    for (; r < r_end; r += kRows * kScaleWarps) {
        float4 part[kRows][S][2];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int row = min(r + i * kScaleWarps, r_end - 1);
#pragma unroll
            for (int q = 0; q < S; ++q)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    part[i][q][c] = peer_load4(peer_smem(sums, q) + row * (4 * kTileCols) + (((32 * c + lane) ^ (row & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int row = r + i * kScaleWarps;
            if (row >= r_end) break;
            float4 v[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                v[c] = part[i][0][c];
#pragma unroll
                for (int q = 1; q < S; ++q) {
                    v[c].x += part[i][q][c].x;
                    v[c].y += part[i][q][c].y;
                    v[c].z += part[i][q][c].z;
                    v[c].w += part[i][q][c].w;
                }
            }
            const int64_t at = (int64_t)(x.m0 + row) * p.N + x.n0 + 4 * lane;
            const int left = p.N - x.n0 - 4 * lane;
            if constexpr (!SWIGLU) {
                store4(p, at, v[0], left);
                store4(p, at + 128, v[1], left - 128);
            } else {   // left is a multiple of 4: N is one of 16
                const float z[4] = {swiglu(v[0].x, v[1].x), swiglu(v[0].y, v[1].y), swiglu(v[0].z, v[1].z),
                                    swiglu(v[0].w, v[1].w)};
                float top = left > 0 ? fmaxf(fmaxf(fabsf(z[0]), fabsf(z[1])), fmaxf(fabsf(z[2]), fabsf(z[3]))) : 0.0f;
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float scale = e4m3_block_scale(top);
                if (lane == 0) p.out_scales[(int64_t)(x.m0 + row) * ((p.N + 127) / 128) + x.n0 / 128] = scale;
                if (left > 0)
                    *reinterpret_cast<uint32_t*>((uint8_t*)p.out + at) =
                        e4m3x4_near(z[0], z[1], z[2], z[3], scale, __frcp_rn(scale));
            }
        }
    }
}

// SPLIT: with SwiGLU, an up block of 128 scales may end inside a tile (N is no multiple of 128).
// KSPLIT: the CTAs of a cluster share one tile, a part of K each, and each finishes a part of its rows.
// TC: columns of a tile, 256 or, with four accumulators and a 16-bit output only, 128.
template <bool SWIGLU, bool SPLIT, bool KSPLIT, int TC>
__global__ void __launch_bounds__(kProductThreads, 1)
ep_product_rows_kernel(const MatmulArgs p, const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b)
{
    static_assert(TC == kTileCols || (TC == 128 && !SWIGLU && !KSPLIT), "the narrow tile is the plain product's");
    constexpr int kStageBytes = stage_bytes(TC), kBuffers = 512 / TC;
    static_assert(kStages % kBuffers == 0, "a stage always goes to the same accumulator");
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 2];
    __shared__ float tops[2][kScaleWarps / 4][kTileRows];   // [tile parity][column half][row]: largest |z|
    __shared__ int4 info[kInfo];              // m0, end of the group's rows, n0 of the tiles being worked on
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
    float* ring = reinterpret_cast<float*>(raw + (stages - smem_u32(raw)) + kStages * kStageBytes);
    int* first = reinterpret_cast<int*>(ring + kRingFloats);
    int32_t* off_copy = first + p.groups + 1;
    const uint32_t full = smem_u32(bars), done = full + 8 * kStages, drained = done + 8 * kStages,
                   topped = drained + 8;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Giveup giveup{&gave_up, p.status};
    constexpr int kCols = SWIGLU ? TC / 2 : TC;   // output columns of a tile
    const int col_tiles = (p.N + kCols - 1) / kCols;
    const int ctas = KSPLIT ? cluster_size() : 1, rank = KSPLIT ? cluster_rank() : 0;
    const int t_first = KSPLIT ? blockIdx.x / ctas : blockIdx.x, t_step = KSPLIT ? gridDim.x / ctas : gridDim.x;
    const int k_lo = KSPLIT ? p.kb * rank / ctas : 0, k_hi = KSPLIT ? p.kb * (rank + 1) / ctas : p.kb;
    const int kb = k_hi - k_lo;   // blocks of this CTA; one at least

    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, 3);   // the loads and two warps' factors
            bar_init(done + 8 * i, 1);
        }
        bar_init(drained, 1);
        bar_init(topped, kScaleWarps);
        fence_barrier_init();
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    if (warp == 2) tmem_alloc(smem_u32(&tmem_slot), 512);
    follow_predecessor();
    const bool copied = p.offsets != nullptr && p.groups <= kSharedOffsets;
    if (copied)
        for (int i = threadIdx.x; i <= p.groups; i += kProductThreads) off_copy[i] = p.offsets[i];
    const int32_t* off = copied ? off_copy : p.offsets;
    if (warp == 1) scan_tiles<kTileRows>(p, first, col_tiles, lane);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_slot;
    // with KSPLIT there is a cluster for every tile, unless the offsets overlap
    const int tiles = uniform(KSPLIT ? min(first[p.groups], t_step) : first[p.groups]);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
            uint32_t n = 0, i = 0;   // blocks loaded, tiles
            const bool leader = elect_one();
            bool ok = true;
            for (int t = t_first; t < tiles && ok; t += t_step, ++i) {
                const Tile x = find_tile<kTileRows, kCols>(p, off, first, col_tiles, t);
                if (leader) {
                    info[i % kInfo] = make_int4(x.m0, x.m1, x.n0, 0);   // seen by whoever sees the block's products
                    const int64_t b_rows = (int64_t)x.g * p.columns;
                    const int y0 = (int)(b_rows + x.n0), y1 = (int)(b_rows + (SWIGLU ? p.N + x.n0 : x.n0 + 128));
                    for (int k = k_lo; k < k_hi; ++k, ++n) {
                        const uint32_t s = n % kStages, use = n / kStages;
                        if (use > 0 && !bar_wait(done + 8 * s, (use - 1) & 1, giveup)) ok = false;
                        if (n == kWithheldBlock || !ok) { ok = false; break; }
                        const uint32_t dst = stages + s * kStageBytes, bar = full + 8 * s;
                        bar_expect(bar, kStageBytes);
                        tma_load(dst, &map_a, k * kBlockK, x.m0, bar);
                        tma_load(dst + kTileRows * kBlockK, &map_b, k * kBlockK, y0, bar);
                        if (TC > 128) tma_load(dst + (kTileRows + 128) * kBlockK, &map_b, k * kBlockK, y1, bar);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            if (leader && !ok) {   // its loads in flight
                const long long t0 = clock64();
                for (uint32_t j = n < kStages ? 0 : n - kStages; j < n; ++j)
                    bar_drain(full + 8 * (j % kStages), (j / kStages) & 1, t0);
            }
            __syncwarp();
        } else if (warp == 1) {
            constexpr uint32_t instruction = mma_instruction(kTileRows, TC);
            const uint64_t a0 = mma_descriptor(stages), b0 = mma_descriptor(stages + kTileRows * kBlockK);
            const uint32_t mine = tiles > t_first ? (tiles - t_first - 1) / t_step + 1 : 0;
            const uint32_t blocks = mine * kb;
            const bool leader = elect_one();
            // after a wait that gave up the products go on, at most kSuspendNs a block, on whatever the stages
            // hold: the scaling warps need every block's arrival
            for (uint32_t n = 0, phase = 0; n < blocks; n += kStages, phase ^= 1) {
#pragma unroll
                for (int s = 0; s < kStages; ++s) {
                    if (n + s >= blocks) break;
                    bar_wait(full + 8 * s, phase, giveup);
                    __syncwarp();
                    if (n + s >= kBuffers) read_wait(s % kBuffers);
                    if (leader) {
                        tmem_fence_after();
#pragma unroll
                        for (int i = 0; i < kBlockK / 32; ++i)
                            mma_e4m3(tmem + (s % kBuffers) * TC, a0 + (s * (kStageBytes >> 4) + 2 * i),
                                     b0 + (s * (kStageBytes >> 4) + 2 * i), instruction, i == 0);
                        mma_commit(done + 8 * s);
                    }
                    __syncwarp();
                }
            }
            for (uint32_t n = blocks < kBuffers ? 0 : blocks - kBuffers; n < blocks; ++n) read_wait(n % kBuffers);
            if (leader) {
                mma_commit(drained);   // tensor memory is freed only after its last product
                bar_drain(drained, 0, clock64());
            }
            __syncwarp();
        } else if (warp >= 2) {
            // factors: as[row][k] * bs[.][k] for rows r and r + 64; loaded kAhead blocks ahead
            const int r = threadIdx.x - 64;
            const int last = p.nb - 1;
            uint32_t n = 0;
            bool ok = true;
            for (int t = t_first; t < tiles && ok; t += t_step) {
                __syncwarp();
                const Tile x = find_tile<kTileRows, kCols>(p, off, first, col_tiles, t);
                const float* as0 = p.as + (int64_t)min(x.m0 + r, x.m1 - 1) * p.kb + k_lo;
                const float* as1 = p.as + (int64_t)min(x.m0 + r + 64, x.m1 - 1) * p.kb + k_lo;
                const float* bs = p.bs + (int64_t)x.g * p.nb * p.kb + k_lo;
                const int up = (SWIGLU ? p.N + x.n0 : x.n0 + 128) / 128;
                const float* bs0 = bs + (int64_t)min(x.n0 / 128, last) * p.kb;
                const float* bs1 = bs + (int64_t)min(up, last) * p.kb;
                const float* bs2 = bs + (int64_t)min(up + 1, last) * p.kb;
                constexpr int kAhead = 4;
                float a0[kAhead], a1[kAhead], b0[kAhead], b1[kAhead], b2[kAhead];
                auto load = [&](int i, int k) {
                    k = min(k, kb - 1);
                    a0[i] = as0[k];
                    a1[i] = as1[k];
                    b0[i] = bs0[k];
                    if (TC > 128) b1[i] = bs1[k];
                    if (SPLIT) b2[i] = bs2[k];
                };
#pragma unroll
                for (int i = 0; i < kAhead; ++i) load(i, i);
                for (int k0 = 0; k0 < kb && ok; k0 += kAhead) {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        if (k0 + i >= kb) break;
                        const uint32_t s = n % kStages, use = n / kStages;
                        // one answer for the warp, whose lanes have to leave together
                        if (use > 0) ok = __all_sync(0xffffffffu, ok && bar_wait(done + 8 * s, (use - 1) & 1, giveup));
                        float* f = ring + (n % kRing) * (kFactors * kTileRows) + r;
                        f[0] = a0[i] * b0[i];
                        f[64] = a1[i] * b0[i];
                        if (TC > 128) {
                            f[kTileRows] = a0[i] * b1[i];
                            f[kTileRows + 64] = a1[i] * b1[i];
                        }
                        if (SPLIT) {
                            f[2 * kTileRows] = a0[i] * b2[i];
                            f[2 * kTileRows + 64] = a1[i] * b2[i];
                        }
                        __syncwarp();
                        if (lane == 0) bar_arrive(full + 8 * s);
                        ++n;
                        load(i, k0 + kAhead + i);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int part = (warp - 4) >> 2;                 // this warp's half of the columns
        const int row = (warp & 3) * 32 + lane;
        // plain: columns part*TC/2 ..; SwiGLU: gate columns part*64 .. (of 128), then their up columns
        const uint32_t col0 = SWIGLU ? part * 64 : part * (TC / 2);
        const uint32_t col1 = SWIGLU ? 128 + part * 64 : col0 + 64;
        // up columns of this part that share a tile's first up block
        const int split = 128 - p.N % 128 - part * 64;
        int parity = 0;
        uint32_t i = 0;
        // of the next block: its products' barrier, that barrier's phase, its accumulator, its factors
        uint32_t next = done, phase = 0, d = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t f = smem_u32(ring) + 4 * (row + (SWIGLU || TC == 128 ? 0 : part * kTileRows));
        const uint32_t f_end = f + kRing * kFactors * kTileRows * 4;
        for (int t = t_first; t < tiles; t += t_step, parity ^= 1, ++i) {
            float2 acc[TC / 4];
#pragma unroll
            for (int j = 0; j < TC / 4; ++j) acc[j] = make_float2(0.0f, 0.0f);
            // another warp's giving up ends nothing here: what follows works on whatever is there, and the rows
            // are not stored
            float f0, f1, f2;
            uint32_t r0[32], r1[32];
            // the block's first columns and its factors, once its products are there
            auto begin = [&](bool ready) {
                if (!ready) products_wait(next, phase, giveup);
                __syncwarp();
                tmem_fence_after();
                tmem_load32(r0, d + col0);
                f0 = smem_load(f);
                f1 = SWIGLU ? smem_load(f + 4 * kTileRows) : f0;
                f2 = SPLIT ? smem_load(f + 8 * kTileRows) : f1;
                next += 8;
                if (next == done + 8 * kStages) { next = done; phase ^= 1; }
                f += 4 * kFactors * kTileRows;
                if (f == f_end) f -= kRing * kFactors * kTileRows * 4;
            };
            begin(false);
            // 32 columns are read while the 32 before them are added, across the ends of blocks too
            for (int k = kb; k > 0; --k) {
                bool ready;
                tmem_wait(r0);
                tmem_load32(r1, d + col0 + 32);
                if constexpr (TC == 128) ready = bar_test(next, phase);
                add_scaled(acc, r0, f0);
                if constexpr (TC > 128) {
                    tmem_wait(r1);
                    tmem_load32(r0, d + col1);
                    ready = bar_test(next, phase);
                    add_scaled(acc + 16, r1, f0);
                    tmem_wait(r0);
                    tmem_load32(r1, d + col1 + 32);
                    if (SPLIT) add_scaled(acc + 32, r0, f1, f2, split);
                    else add_scaled(acc + 32, r0, f1);
                }
                tmem_wait(r1);
                tmem_fence_before();
                read_arrive((d & 511) / TC);   // tensor memory starts at column 0: it is allocated whole
                d = (d & ~511u) | ((d + TC) & 511);
                const float g1 = TC > 128 ? f1 : f0, g2 = f2;
                if (k > 1) begin(ready);
                if (SPLIT) add_scaled(acc + TC / 4 - 16, r1, g1, g2, split - 32);
                else add_scaled(acc + TC / 4 - 16, r1, g1);
            }
            const int4 x = info[i % kInfo];
            if constexpr (KSPLIT) {
                // the cluster's only tile: every load has arrived and been multiplied, so the stages hold the
                // sums, [row][256 columns], 16-byte pieces exchanged so that neither side meets a bank twice
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const uint32_t piece = ((j < 16 ? col0 : col1 - 64) >> 2) + j;
                    smem_store4(stages + row * (4 * kTileCols) + ((piece ^ (row & 7)) << 4), acc[2 * j], acc[2 * j + 1]);
                }
            } else if constexpr (!SWIGLU) {
                const int n0 = x.z + part * (TC / 2), m = x.y - x.x - (warp & 3) * 32;   // rows of this warp's 32 that exist
                const int64_t pitch = 2 * (int64_t)p.N;
                uint8_t* out = (uint8_t*)p.out + (int64_t)(x.x + (warp & 3) * 32) * pitch + 2 * n0;
                if (!__any_sync(0xffffffffu, *giveup.flag) && n0 < p.N) {
                    if (p.dtype == EP_FP16) store_rows<true, TC / 4>(out, pitch, acc, m, p.N - n0, p.vec);
                    else store_rows<false, TC / 4>(out, pitch, acc, m, p.N - n0, p.vec);
                }
            } else {
                const int n0 = x.z + part * 64;
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    acc[j].x = swiglu(acc[j].x, acc[32 + j].x);
                    acc[j].y = swiglu(acc[j].y, acc[32 + j].y);
                    if (!SPLIT || n0 + 2 * j < p.N) top = fmaxf(top, fmaxf(fabsf(acc[j].x), fabsf(acc[j].y)));
                }
                tops[parity][part][row] = top;
                // the other part's maximum; a parity's words are rewritten two tiles later, which no warp
                // reaches before all have passed the tile between
                __syncwarp();
                if (lane == 0) bar_arrive(topped);
                const bool ok = bar_wait(topped, parity, giveup) && !*giveup.flag;
                const float scale = e4m3_block_scale(fmaxf(top, tops[parity][part ^ 1][row]));
                const float inv = __frcp_rn(scale);
                if (ok && x.x + row < x.y) {
                    if (part == 0) p.out_scales[(int64_t)(x.x + row) * ((p.N + 127) / 128) + x.z / 128] = scale;
                    uint8_t* out = (uint8_t*)p.out + (int64_t)(x.x + row) * p.N + n0;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t c[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            c[j] = e4m3x4_near(acc[16 * b + 2 * j].x, acc[16 * b + 2 * j].y, acc[16 * b + 2 * j + 1].x,
                                               acc[16 * b + 2 * j + 1].y, scale, inv);
                        const uint4 lo = make_uint4(c[0], c[1], c[2], c[3]), hi = make_uint4(c[4], c[5], c[6], c[7]);
                        const int left = p.N - n0 - 32 * b;   // columns; a multiple of 16
                        if (p.vec == 2 && left >= 32) {
                            st_v8(out + 32 * b, lo, hi);
                        } else {
                            if (left > 0) st_v4(out + 32 * b, lo);
                            if (left > 16) st_v4(out + 32 * b + 16, hi);
                        }
                    }
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if constexpr (KSPLIT) {
        cluster_sync();   // the sums of every CTA are there
        if (warp >= 4 && t_first < tiles && !gave_up) {
            const Tile x = find_tile<kTileRows, kCols>(p, off, first, col_tiles, t_first);   // whole warps
            const int per = kTileRows / ctas;   // rows this CTA finishes, a warp every eighth
            const int r = rank * per + warp - 4, r_end = min((rank + 1) * per, x.m1 - x.m0);
            if (ctas == 2) finish_rows<SWIGLU, 2>(p, x, stages, r, r_end);
            else if (ctas == 4) finish_rows<SWIGLU, 4>(p, x, stages, r, r_end);
            else finish_rows<SWIGLU, 8>(p, x, stages, r, r_end);
        }
        cluster_sync();   // every CTA has taken what it needs of this one's sums
    }
    if (warp == 2) {
        tmem_fence_after();
        tmem_free(tmem, 512);
    }
}

// ---- few rows
//
// With few rows to a group the time is that of reading b once.  Here b's rows are the 128 lanes of the
// accumulator and the T rows of a tile, 16 or 32, its columns: a CTA takes 128 output columns (with
// SwiGLU also their 128 up rows) and T rows, and streams b through as many stages as shared memory holds
// (about 180 KB in flight on an SM; the rows' codes come from L2).  Tiles are small enough to spread the
// weights evenly, and where there are too few of them for the SMs a cluster of CTAs splits K: each
// leaves its sums in its shared memory, and each adds up, in the order of the CTAs, the rows of T
// that it finishes.  Roles as above, with four scaling warps: a thread owns one output column.
//
// 256 rows in 32 groups, 7168 x 4096 with SwiGLU: 143 us, 6.6 TB/s (0.97 of the measured copy), tensor cores
// 4 % busy.  One row of 7168 x 2048: 6 us where the weights' bytes take 2.2; the rest is the launch, the
// first load's way from HBM and the cluster's exchange, each 1 to 2 us.

constexpr int kFewThreads = 256;
constexpr int kFewCols = 128;
constexpr int kFewRing = 16;          // blocks of factors: at least stages + accumulators
constexpr int kFewMaxStages = 12;
constexpr int kFewReadThreads = 128 + 32;

template <int T, bool SWIGLU>
struct FewShape {
    static constexpr int kHalves = SWIGLU ? 2 : 1;
    static constexpr int kWeightBytes = kFewCols * kBlockK;
    static constexpr int kStageBytes = kHalves * kWeightBytes + T * kBlockK;
    static constexpr int kBufferCols = kHalves * T;
    // accumulators: no more than stages, so that a stage's barrier is never a whole phase ahead of a reader
    static constexpr int kBuffers = 4;
    static constexpr int kTmemCols = kBuffers * kBufferCols < 32 ? 32 : kBuffers * kBufferCols;
    static constexpr int kFactorRows = SWIGLU ? 3 : 1;   // gate, and the two up blocks a tile can touch
    static constexpr int kRingFloats = kFewRing * kFactorRows * T;
    static constexpr int kSumFloats = kHalves * T * kFewCols;
};

template <int T, bool SWIGLU>
__global__ void __launch_bounds__(kFewThreads, 1)
ep_product_few_kernel(const MatmulArgs p, const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b, const int stage_count, const int split_k)
{
    using S = FewShape<T, SWIGLU>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * kFewMaxStages + 3];
    __shared__ float tops[2][4][T];   // [tile parity][warp][row]: largest |z|
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
    float* sums = reinterpret_cast<float*>(raw + (stages - smem_u32(raw)) + stage_count * S::kStageBytes);
    float* ring = sums + S::kSumFloats;
    int* first = reinterpret_cast<int*>(ring + S::kRingFloats);
    int32_t* off_copy = first + p.groups + 1;
    const uint32_t full = smem_u32(bars), done = full + 8 * kFewMaxStages, drained = done + 8 * kFewMaxStages,
                   summed = drained + 8, taken = summed + 8;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Giveup giveup{&gave_up, p.status};
    const int col_tiles = (p.N + kFewCols - 1) / kFewCols;
    const uint32_t rank = split_k > 1 ? cluster_rank() : 0;
    const int k_lo = (int)((int64_t)p.kb * rank / split_k), k_hi = (int)((int64_t)p.kb * (rank + 1) / split_k);
    const int t_first = blockIdx.x / split_k, t_step = gridDim.x / split_k;

    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < stage_count; ++i) {
            bar_init(full + 8 * i, 3);   // the loads and two warps' factors
            bar_init(done + 8 * i, 1);
        }
        bar_init(drained, 1);
        bar_init(summed, 4 * split_k);
        bar_init(taken, 4 * split_k);
        fence_barrier_init();
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    if (warp == 2) tmem_alloc(smem_u32(&tmem_slot), S::kTmemCols);
    follow_predecessor();
    const bool copied = p.offsets != nullptr && p.groups <= kSharedOffsets;
    if (copied)
        for (int i = threadIdx.x; i <= p.groups; i += kFewThreads) off_copy[i] = p.offsets[i];
    const int32_t* off = copied ? off_copy : p.offsets;
    if (warp == 1) scan_tiles<T>(p, first, col_tiles, lane);
    tmem_fence_before();
    __syncthreads();
    if (split_k > 1) cluster_sync();   // the peers' barriers exist
    tmem_fence_after();
    const uint32_t tmem = tmem_slot;
    const int tiles = uniform(first[p.groups]);

    if (warp == 0) {
        uint32_t n = 0, s = 0, phase = 1;
        const bool leader = elect_one();
        bool ok = true;
        for (int t = t_first; t < tiles && ok; t += t_step) {
            const Tile x = find_tile<T, kFewCols>(p, off, first, col_tiles, t);
            if (leader) {
                const int y = (int)((int64_t)x.g * p.columns + x.n0);
                for (int k = k_lo; k < k_hi; ++k, ++n) {
                    if (n >= (uint32_t)stage_count && !bar_wait(done + 8 * s, phase, giveup)) ok = false;
                    if (n == kWithheldBlock || !ok) { ok = false; break; }
                    const uint32_t dst = stages + s * S::kStageBytes, bar = full + 8 * s;
                    bar_expect(bar, S::kStageBytes);
                    tma_load(dst, &map_b, k * kBlockK, y, bar);
                    if (SWIGLU) tma_load(dst + S::kWeightBytes, &map_b, k * kBlockK, y + p.N, bar);
                    tma_load(dst + S::kHalves * S::kWeightBytes, &map_a, k * kBlockK, x.m0, bar);
                    if (++s == (uint32_t)stage_count) { s = 0; phase ^= 1; }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        if (leader && !ok) {   // its loads in flight
            const long long t0 = clock64();
            for (uint32_t i = n < (uint32_t)stage_count ? 0 : n - stage_count; i < n; ++i)
                bar_drain(full + 8 * (i % stage_count), (i / stage_count) & 1, t0);
        }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t instruction = mma_instruction(kFewCols, T);
        const uint64_t d0 = mma_descriptor(stages);
        const uint32_t mine = tiles > t_first ? (tiles - t_first - 1) / t_step + 1 : 0;
        const uint32_t blocks = mine * (k_hi - k_lo);
        const bool leader = elect_one();
        // after a wait that gave up the products go on, on whatever the stages hold (see above)
        for (uint32_t n = 0, s = 0, phase = 0; n < blocks; ++n) {
            const uint32_t buf = n % S::kBuffers;
            bar_wait(full + 8 * s, phase, giveup);
            __syncwarp();
            if (n >= S::kBuffers) asm volatile("bar.sync %0, %1;" :: "r"(1 + buf), "n"(kFewReadThreads) : "memory");
            if (leader) {
                tmem_fence_after();
                const uint64_t w = d0 + s * (uint32_t)(S::kStageBytes >> 4);
                const uint64_t r = w + S::kHalves * (S::kWeightBytes >> 4);
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                    for (int i = 0; i < kBlockK / 32; ++i)
                        mma_e4m3(tmem + buf * S::kBufferCols + h * T, w + h * (S::kWeightBytes >> 4) + 2 * i, r + 2 * i,
                                 instruction, i == 0);
                mma_commit(done + 8 * s);
            }
            __syncwarp();
            if (++s == (uint32_t)stage_count) { s = 0; phase ^= 1; }
        }
        for (uint32_t n = blocks < S::kBuffers ? 0 : blocks - S::kBuffers; n < blocks; ++n)
            asm volatile("bar.sync %0, %1;" :: "r"(1 + n % S::kBuffers), "n"(kFewReadThreads) : "memory");
        if (leader) {
            mma_commit(drained);   // tensor memory is freed only after its last product
            bar_drain(drained, 0, clock64());
        }
        __syncwarp();
    } else if (warp < 4) {
        // factors of row c of the tile: as[row][k] * bs[.][k]; loaded kAhead blocks ahead
        const int c = threadIdx.x - 64;
        const int last = p.nb - 1;
        uint32_t n = 0, s = 0, phase = 1;
        bool ok = true;
        for (int t = t_first; t < tiles && ok; t += t_step) {
            __syncwarp();
            const Tile x = find_tile<T, kFewCols>(p, off, first, col_tiles, t);
            const float* as = p.as + (int64_t)min(x.m0 + c, x.m1 - 1) * p.kb;
            const float* bs = p.bs + (int64_t)x.g * p.nb * p.kb;
            const int up = (p.N + x.n0) / 128;
            const float* bs0 = bs + (int64_t)min(x.n0 / 128, last) * p.kb;
            const float* bs1 = bs + (int64_t)min(up, last) * p.kb;
            const float* bs2 = bs + (int64_t)min(up + 1, last) * p.kb;
            constexpr int kAhead = 4;
            float a[kAhead], b0[kAhead], b1[kAhead], b2[kAhead];
            auto load = [&](int i, int k) {
                if (c >= T || k >= k_hi) return;
                a[i] = as[k];
                b0[i] = bs0[k];
                if (SWIGLU) { b1[i] = bs1[k]; b2[i] = bs2[k]; }
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load(i, k_lo + i);
            for (int k0 = k_lo; k0 < k_hi && ok; k0 += kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (k0 + i >= k_hi) break;
                    // one answer for the warp, whose lanes have to leave together
                    if (n >= (uint32_t)stage_count) ok = __all_sync(0xffffffffu, ok && bar_wait(done + 8 * s, phase, giveup));
                    if (c < T) {
                        float* f = ring + (n % kFewRing) * (S::kFactorRows * T) + c;
                        f[0] = a[i] * b0[i];
                        if (SWIGLU) { f[T] = a[i] * b1[i]; f[2 * T] = a[i] * b2[i]; }
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(full + 8 * s);
                    ++n;
                    if (++s == (uint32_t)stage_count) { s = 0; phase ^= 1; }
                    load(i, k0 + kAhead + i);
                }
            }
        }
    } else {
        const int col = threadIdx.x - 128;
        const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t my_sums = smem_u32(sums) + 4 * col;
        bool ok = true;
        uint32_t n = 0, s = 0, phase = 0, parity = 0;
        const int c_lo = T * rank / split_k, c_hi = T * (rank + 1) / split_k;   // the rows this CTA finishes
        for (int t = t_first; t < tiles; t += t_step, parity ^= 1) {
            __syncwarp();
            const Tile x = find_tile<T, kFewCols>(p, off, first, col_tiles, t);
            const int up_row = (p.N + x.n0 + col) / 128 - (p.N + x.n0) / 128;   // 0 or 1: this column's up block
            float2 acc[S::kHalves][T / 2];
#pragma unroll
            for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                for (int i = 0; i < T / 2; ++i) acc[h][i] = make_float2(0.0f, 0.0f);
            for (int k = k_lo; k < k_hi; ++k, ++n) {
                const uint32_t buf = n % S::kBuffers;
                products_wait(done + 8 * s, phase, giveup);
                tmem_fence_after();
                const float* f = ring + (n % kFewRing) * (S::kFactorRows * T);
#pragma unroll
                for (int h = 0; h < S::kHalves; ++h) {
                    const float* fh = f + (h ? (1 + up_row) * T : 0);
#pragma unroll
                    for (int i = 0; i < T; i += 16) {
                        uint32_t r[16];
                        tmem_load16(r, taddr + buf * S::kBufferCols + h * T + i);
                        tmem_wait(r);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(fh + i + j);
                            fma2(acc[h][(i + j) / 2], make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                 make_float2(v.x, v.y));
                            fma2(acc[h][(i + j) / 2 + 1],
                                 make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), make_float2(v.z, v.w));
                        }
                    }
                }
                tmem_fence_before();
                asm volatile("bar.arrive %0, %1;" :: "r"(1 + buf), "n"(kFewReadThreads) : "memory");
                if (++s == (uint32_t)stage_count) { s = 0; phase ^= 1; }
            }
            // this CTA's sums; before they are replaced every CTA has taken the last tile's
            if (split_k > 1 && t != t_first) ok &= peer_wait(taken, parity ^ 1, giveup);
#pragma unroll
            for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
                for (int i = 0; i < T / 2; ++i) {
                    sums[(h * T + 2 * i) * kFewCols + col] = acc[h][i].x;
                    sums[(h * T + 2 * i + 1) * kFewCols + col] = acc[h][i].y;
                }
            if (split_k > 1) {
                __syncwarp();
                if (lane < split_k) peer_arrive(peer_smem(summed, lane));
                ok &= peer_wait(summed, parity, giveup);
            }
            auto total = [&](int j) {   // sums of row j (of gate rows, then up rows) over the cluster
                if (split_k == 1) return sums[j * kFewCols + col];
                float part[kMaxSplit], v = 0.0f;   // all loads on their way before the first is added
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q)
                    part[q] = q < split_k ? peer_load(peer_smem(my_sums + j * kFewCols * 4, q)) : 0.0f;
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q) v += part[q];
                return v;
            };
            const int rows = min(x.m1 - x.m0, c_hi);
            const bool in = x.n0 + col < p.N;
            if constexpr (!SWIGLU) {
                for (int c = c_lo; c < rows; ++c) {
                    const float v = total(c);
                    if (!ok || !in) continue;
                    const int64_t at = (int64_t)(x.m0 + c) * p.N + x.n0 + col;
                    if (p.dtype == EP_FP16) ((__half*)p.out)[at] = __float2half_rn(v);
                    else ((__nv_bfloat16*)p.out)[at] = __float2bfloat16_rn(v);
                }
            } else {
                for (int c = c_lo; c < rows; ++c) {
                    const float gate = total(c), up = total(T + c);
                    const float z = swiglu(gate, up);
                    sums[c * kFewCols + col] = z;   // only this thread reads it from now on
                    // whole-number order is that of magnitudes; fmaxf turns NaN into 0
                    const unsigned top = __reduce_max_sync(0xffffffffu, __float_as_uint(in ? fmaxf(fabsf(z), 0.0f) : 0.0f));
                    if (lane == 0) tops[parity][warp & 3][c] = __uint_as_float(top);
                }
                asm volatile("bar.sync 7, 128;" ::: "memory");
                for (int c = c_lo; c < rows; ++c) {
                    const float* w = &tops[parity][0][c];
                    const float scale = e4m3_block_scale(fmaxf(fmaxf(w[0], w[T]), fmaxf(w[2 * T], w[3 * T])));
                    if (!ok) continue;
                    if (col == 0) p.out_scales[(int64_t)(x.m0 + c) * ((p.N + 127) / 128) + x.n0 / 128] = scale;
                    if (in)
                        ((uint8_t*)p.out)[(int64_t)(x.m0 + c) * p.N + x.n0 + col] =
                            (uint8_t)e4m3x2(near_quotient(sums[c * kFewCols + col], scale, __frcp_rn(scale)), 0.0f);
                }
            }
            if (split_k > 1) {
                __syncwarp();
                if (lane < split_k) peer_arrive(peer_smem(taken, lane));
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (split_k > 1) cluster_sync();
    if (warp == 2) {
        tmem_fence_after();
        tmem_free(tmem, S::kTmemCols);
    }
}

// ---- tensor maps

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (EncodeTiled)f;
    }();
    return fn;
}

// Map of [rows][K] codes with boxes of box_rows x 128 bytes, swizzled by 128 bytes; elements past either
// end read as zero codes.
int make_map(CUtensorMap* m, const char* what, const void* base, int64_t rows, int K, int box_rows)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return layer_fail(EP_ERR_CUDA, "ep_matmul_fp8: the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, pitch[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {kBlockK, (cuuint32_t)box_rows}, step[2] = {1, 1};
    auto make = [&] {
        return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, pitch, box, step,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = make();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {   // a host thread's first call, which nothing has bound to the device yet
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaSetDevice(dev);
        if (e != cudaSuccess) return layer_cuda(e, "ep_matmul_fp8: binding the host thread to its device");
        r = make();
    }
    if (r != CUDA_SUCCESS) return layer_fail(EP_ERR_CUDA, "ep_matmul_fp8: tensor map of %s: CUresult %d", what, (int)r);
    return EP_OK;
}

template <typename... Params, typename... Args>
cudaError_t launch_cluster(void (*k)(Params...), unsigned grid, int threads, size_t smem, int ctas, cudaStream_t s,
                           const Args&... args)   // launch_dependent with clusters of `ctas`
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

// Tiles, at most, of `rows` rows in groups: every group that holds a row can end inside a tile.
int64_t most_tiles(const MatmulArgs& p, int rows, int cols)
{
    const int64_t groups = p.groups < p.rows ? p.groups : p.rows;
    return ((p.rows - groups) / rows + groups) * ((p.N + cols - 1) / cols);
}

// CTAs that share a tile's K, each at least `least` blocks: 1, 2 or 4 while they fit the SMs; 8 only for a few
// tiles, because a GPC's 16 to 20 SMs hold two clusters of 8 at most and 16 clusters do not all run at once
// (one row, 7168 x 4096 with SwiGLU: 13.7 us in 8, 9.2 in 4, 13.1 in 2).
int split_of(const MatmulArgs& p, int64_t tiles, int least, int sms)
{
    int split = 1;
    while (split < (tiles <= 8 ? kMaxSplit : 4) && tiles * split * 2 <= sms && split * 2 * least <= p.kb) split *= 2;
    return split;
}

template <auto* K>
cudaError_t launch_tiles(const MatmulArgs& p, const CUtensorMap& ma, const CUtensorMap& mb, int stage, int64_t tiles,
                         int split, int sms, cudaStream_t s)
{
    const size_t smem = 1024 + kStages * stage + kRingFloats * sizeof(float) + (p.groups + 1) * sizeof(int) +
                        (p.offsets && p.groups <= kSharedOffsets ? (p.groups + 1) * sizeof(int32_t) : 0);
    const cudaError_t e = allow_all_shared<K>();
    if (e != cudaSuccess) return e;
    const int64_t grid = split > 1 ? tiles * split : tiles < sms ? tiles : sms;
    return launch_cluster(K, (unsigned)grid, kProductThreads, smem, split, s, p, ma, mb);
}

template <bool SWIGLU, bool SPLIT>
cudaError_t launch_product_rows(const MatmulArgs& p, const CUtensorMap& ma, const CUtensorMap& mb, int sms,
                                cudaStream_t s)
{
    const int64_t most = most_tiles(p, kTileRows, SWIGLU ? kTileCols / 2 : kTileCols);
    // The sums' exchange costs what half a dozen blocks do.  256 rows, us, whole against shared: 7168 x 2048
    // 22.1 : 12.8 in 4, 4096 x 1024 14.2 : 10.6 in 4, 2048 x 7168 (16 blocks) 9.4 : 10.8 in 2.
    const int split = p.kb < kSharedBlocks ? 1 : split_of(p, most, 7, sms);
    // Half as wide while the tiles still fit the SMs at once, which shortens a tile's blocks and its end.  us, 256
    // against 128 columns: 200 rows of 2048 x 2048 9.2 : 6.3, 1777 rows of 1040 x 520 in 6 groups 10.4 : 7.9; past
    // the SMs, 512 rows of 2048 x 7168 (112 : 224 tiles) 11.0 : 12.2.
    const int64_t narrow = most_tiles(p, kTileRows, 128);
    if (!SWIGLU && split == 1 && narrow <= sms)
        return launch_tiles<ep_product_rows_kernel<false, false, false, 128>>(p, ma, mb, stage_bytes(128), narrow, 1, sms, s);
    constexpr int kStage = stage_bytes(kTileCols);
    if (split > 1)
        return launch_tiles<ep_product_rows_kernel<SWIGLU, SPLIT, true, kTileCols>>(p, ma, mb, kStage, most, split, sms, s);
    return launch_tiles<ep_product_rows_kernel<SWIGLU, SPLIT, false, kTileCols>>(p, ma, mb, kStage, most, 1, sms, s);
}

template <int T, bool SWIGLU>
cudaError_t launch_product_few(const MatmulArgs& p, const CUtensorMap& ma, const CUtensorMap& mb, int sms,
                               cudaStream_t s)
{
    using S = FewShape<T, SWIGLU>;
    const int64_t most = most_tiles(p, T, kFewCols);
    const int split = split_of(p, most, 1, sms);
    const size_t rest = 1024 + (S::kSumFloats + S::kRingFloats) * sizeof(float) + (p.groups + 1) * sizeof(int) +
                        (p.offsets && p.groups <= kSharedOffsets ? (p.groups + 1) * sizeof(int32_t) : 0);
    constexpr size_t kMost = 227 * 1024 - 4096;   // less the static part
    int stages = (int)((kMost - rest) / S::kStageBytes);
    if (stages > kFewMaxStages) stages = kFewMaxStages;
    if (stages < S::kBuffers) return cudaErrorInvalidConfiguration;   // not reached: 4 stages at the least
    const size_t smem = rest + (size_t)stages * S::kStageBytes;
    const cudaError_t e = allow_all_shared<ep_product_few_kernel<T, SWIGLU>>();
    if (e != cudaSuccess) return e;
    const int64_t clusters = most < sms / split ? most : sms / split;
    return launch_cluster(ep_product_few_kernel<T, SWIGLU>, (unsigned)(clusters * split), kFewThreads, smem, split, s, p,
                          ma, mb, stages, split);
}

// Rows of a tile of the kernel for few rows, or 0 for the kernel of 128-row tiles.  Measured, us, few rows
// against 128-row tiles:
//   one group, 7168 x 4096 with SwiGLU   1 row 8.5 : 11.9   32 rows 11.0 : 13.2   64 rows 12.9 : 13.5   96 rows 18.3 : 13.9
//   one group, 2048 x 2048               1 row 4.6 : 5.7    32 rows 5.8 : 5.9     64 rows 6.9 : 5.9
//   one group, 1024 x 1024               1 row 4.3 : 4.2    32 rows 5.1 : 4.3
//   4 groups, 7168 x 2048                of 4 rows 14.8 : 16.4   of 8 rows 16.1 : 15.7   of 16 rows 18.8 : 16.5
//   32 groups, 7168 x 4096 with SwiGLU   of 8 rows 145 : 152     of 16 rows 152 : 153    of 24 rows 167 : 153
// The 128-row tiles multiply rows that are not there, which costs them nothing while the weights' bytes or
// the tiles' number set the time; a group whose rows pass a tile of few reads its weights twice.
// The host knows p.rows alone, not what the groups hold of them: a buffer far longer than its groups takes the
// 128-row tiles (256 rows held of 262144, 32 groups, 7168 x 4096 with SwiGLU 151 us, against 143 in a buffer of
// their length; 8 rows held 36.4 against 32.8; 256 held of 32768, 2048 x 7168 73 against 75).
int few_rows_tile(const MatmulArgs& p, int sms)
{
    // whether the wide tiles leave half of the SMs to narrower ones or to parts of K
    const bool idle = 2 * most_tiles(p, kTileRows, p.swiglu ? kTileCols / 2 : kTileCols) <= sms;
    if (p.groups == 1) {
        if (p.rows > 64 || (p.kb <= 8 && (!p.swiglu || p.rows > 32))) return 0;
        if (p.rows <= 32) return 16;
        return !p.swiglu && p.kb < kSharedBlocks && idle ? 0 : 32;
    }
    const int64_t groups = p.groups < p.rows ? p.groups : p.rows;   // that can hold a row
    const int64_t mean = p.rows / groups;
    return mean < 8 || (mean == 8 && !idle) ? 16 : mean <= 16 && !idle ? 32 : 0;
}

}  // namespace
}  // namespace ep

extern "C" int ep_matmul_fp8(const void* a, const float* a_scales, const void* b, const float* b_scales,
                             const int32_t* offsets, int64_t rows, int groups, int columns, int inner, int swiglu,
                             int dtype, void* out, float* out_scales, int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_matmul_fp8";
    if (rows < 0 || rows > INT32_MAX - kTileRows)   // a tile's last row is counted in 32 bits
        return layer_fail(EP_ERR_ARG, "%s: rows=%lld outside 0..2^31-1-%d", who, (long long)rows, kTileRows);
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
    p.columns = columns;
    p.vec = swiglu ? (p.N % 32 == 0 && layer_aligned(out, 32) ? 2 : 1)
                   : columns % 16 == 0 && layer_aligned(out, 32) ? 2 : columns % 8 == 0 ? 1 : 0;
    const int sms = layer_num_sms();
    if (sms == 0) return layer_fail(EP_ERR_CUDA, "%s: cannot tell the current device's multiprocessors", who);
    // rows of a tile of the kernel for few rows, or 0 for the kernel of 128-row tiles
    const int few = few_rows_tile(p, sms);
    CUtensorMap ma, mb;
    if (int rc = make_map(&ma, "a", a, rows, inner, few ? few : kTileRows)) return rc;
    if (int rc = make_map(&mb, "b", b, (int64_t)groups * columns, inner, 128)) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (few == 16)
        e = swiglu ? launch_product_few<16, true>(p, ma, mb, sms, s) : launch_product_few<16, false>(p, ma, mb, sms, s);
    else if (few == 32)
        e = swiglu ? launch_product_few<32, true>(p, ma, mb, sms, s) : launch_product_few<32, false>(p, ma, mb, sms, s);
    else if (!swiglu) e = launch_product_rows<false, false>(p, ma, mb, sms, s);
    else if (p.N % 128 == 0) e = launch_product_rows<true, false>(p, ma, mb, sms, s);
    else e = launch_product_rows<true, true>(p, ma, mb, sms, s);
    return layer_cuda(e, "ep_matmul_fp8: launch");
}
