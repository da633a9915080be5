// ep_wgrad.cu -- gradient of the block-scaled product for its weights, from rows kept as e4m3 codes.
//
//   dw[g][n][k] = sum over the rows i of group g of  dy[i][n] * (a[i][k] * a_scales[i][k / 128])
//
// on the 16-bit tensor cores: dy as it is, a's values rounded once to dy's type on their way (half a unit of 8 bits, or of
// 11 with FP16, in each term of a sum in FP32), the result rounded once.  The scales differ from row to row, that is along
// the sum, so they cannot enter after the product.
//
// Both operands lie in memory as rows, and the sum runs over rows: each is read as it lies, lines of 64 columns with K
// from line to line.  A pair of CTAs makes tiles of 256 columns of dy by 256 of a; each holds 128 columns of either
// operand and 128 x 256 sums in tensor memory, twice, so that a tile's sums leave while the next is multiplied.  Per CTA:
// warp 0 loads 64 rows of dy and of codes by TMA, and the rows' scales, into one of kGradStages stages; two warps to a
// stage make 16-bit values of the codes, in the order that the tensor cores read; warp 1 of the first CTA multiplies for
// both; eight warps hand the sums to TMA stores.
//
// Measured: 8192 rows in 8 groups of 4096 x 7168 317 us in a burst (1520 TFLOP/s), 2048 in 16 groups 171 us (5.5 TB/s of
// dw), 32768 in 32 groups 1240 us in a burst and 1397 to 1433 at the power limit (1340 to 1380 TFLOP/s at 1.75 GHz; a plain
// BF16 product reaches 1890 in a burst and 1700 at the limit); with FP32 sums out 347, 318 and 1365 to 1531.  A stage takes 850
// cycles, of which its products need 512 and shared memory 640: 24 KB come in, the codes are read, the values written, and the
// tensor cores read 32 KB.  The rest is the conversion, a stage's chain of 128 codes a lane: with it left out, and the sums' way
// out as it was before, 340 us became 259.
//
// A pair sums all rows of its tile, so fewer tiles than half the SMs leave SMs idle: 16384 rows into 1024 x 1024, 512 x 512 and
// 136 x 256 take 86, 85 and 83 us, 256 stages one after another, where bytes and operations take 18, 5 and 1.
#include "ep_tcgen05.cuh"

namespace ep {
namespace {

constexpr int kGradRows = 64;                      // of a stage
constexpr int kGradHalf = 128;                     // columns of either operand in a CTA
constexpr int kGradTile = 2 * kGradHalf;
constexpr int kLineBytes = 8192;                   // 64 columns x 64 rows of 16 bits
constexpr int kDyBytes = 2 * kLineBytes, kValueBytes = 2 * kLineBytes, kCodeBytes = kGradRows * kGradHalf;
constexpr int kGradStageBytes = kDyBytes + kValueBytes + kCodeBytes;
constexpr int kGradStages = 5;
// Two to a quarter of the lanes, 128 columns each.  8 and 4 warps: 8192 rows in 8 groups of 4096 x 7168 314 and 320 us, 2048
// in 16 groups 171 and 226 (before pair_arrive's fence, which adds 1 to 2 %, as below).
constexpr int kWriteWarps = 8;
constexpr int kFirstWriter = 2, kFirstConverter = kFirstWriter + kWriteWarps;
// Warps that convert a stage.  Each stage has a team of its own: a barrier's parity tells one phase from the next alone, so
// whoever waits for a stage's phase has to have seen the one before.  Teams of 2 and 4 warps: the same rows
// 314 and 341 us, 171 and 182 (with 62 registers a thread instead of 93); of 1 against 2, when both were slower, 401 and 352.
constexpr int kConvertTeam = 2;
constexpr int kGradThreads = 32 * (kFirstConverter + kGradStages * kConvertTeam);   // load, multiply, write, convert
constexpr int kMaxGradGroups = 4096;
constexpr int kOutBytes = 2048;   // of a writing warp
// A tile's sums come after all of its stages, up to 2^25 of some 850 cycles: the wait for them is given this much for each.
constexpr long long kStageCycles = 1 << 13;
constexpr size_t kGradShared = 1024 + kGradStages * (kGradStageBytes + kGradRows * 4) + kWriteWarps * kOutBytes;

struct GradArgs {
    const float* a_scales;
    const int32_t* offsets;   // [groups + 1], or NULL: one group of all rows
    int* status;
    int64_t rows;
    int groups, columns, inner, kb;
    int n_tiles, k_tiles;
    int64_t tiles;
    int out_fp32;
};

struct GradTile {
    int g, n0, k0, r0, r1;
};

__device__ __forceinline__ GradTile grad_tile(const GradArgs& p, int64_t t)
{
    GradTile x;
    const int per = p.n_tiles * p.k_tiles;
    x.g = (int)(t / per);
    const int in = (int)(t - (int64_t)x.g * per);
    x.n0 = in / p.k_tiles * kGradTile;
    x.k0 = in % p.k_tiles * kGradTile;
    x.r0 = 0;
    x.r1 = (int)p.rows;
    if (p.offsets) {
        x.r0 = max(0, min(p.offsets[x.g], (int)p.rows));
        x.r1 = max(x.r0, min(p.offsets[x.g + 1], (int)p.rows));
    }
    return x;
}

__device__ __forceinline__ int grad_steps(const GradTile& x) { return (x.r1 - x.r0 + kGradRows - 1) / kGradRows; }

// A warp's 32 rows of 32 sums to memory, through 2 KB of shared memory of its own and a TMA store, which writes no more
// of them than exist: x and y are their first column and row in group g.  32-bit sums go in two halves.  The box's rows
// of 64 bytes are swizzled, so that eight lanes' 16 bytes fill all banks.
template <bool FP16>
__device__ __forceinline__ void write_sums(const GradArgs& p, const CUtensorMap* map, uint32_t buffer, const uint32_t (&r)[32],
                                           int x, int y, int g)
{
    const int lane = threadIdx.x & 31;
    auto send = [&](const uint32_t* w, int column) {
        if (lane == 0) stores_wait_read();   // of what was in the buffer
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            smem_store4(buffer + 64 * lane + ((j ^ ((lane >> 1) & 3)) << 4), make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
        fence_async();
        __syncwarp();
        if (lane == 0) tma_store3(map, buffer, column, y, g);
    };
    if (p.out_fp32) {
        send(r, x);
        if (x + 16 < p.inner) send(r + 16, x + 16);
    } else {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack2<FP16>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        send(w, x);
    }
}

template <bool FP16>
__global__ void __launch_bounds__(kGradThreads, 1)
ep_weight_gradient_kernel(const GradArgs p, const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_a,
                          const __grid_constant__ CUtensorMap map_dw)
{
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[5 * kGradStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u, outs = stages + kGradStages * kGradStageBytes,
                   scales = outs + kWriteWarps * kOutBytes;
    // coded: a stage's codes and scales are here; taken: they have been converted; loaded: its rows of dy are here; ready (the
    // first CTA's): both CTAs' operands are; done: its products are
    const uint32_t coded = smem_u32(bars), taken = coded + 8 * kGradStages, loaded = taken + 8 * kGradStages,
                   ready = loaded + 8 * kGradStages, done = ready + 8 * kGradStages, summed = done + 8 * kGradStages,
                   written = summed + 16, drained = written + 16;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Giveup giveup{&gave_up, p.status};
    const int rank = (int)cluster_rank();
    const int64_t t_first = blockIdx.x / 2, t_step = gridDim.x / 2;

    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kGradStages; ++i) {
            bar_init(coded + 8 * i, 1 + 32);
            bar_init(taken + 8 * i, kConvertTeam);
            bar_init(loaded + 8 * i, 1);
            bar_init(ready + 8 * i, 2 * kConvertTeam);
            bar_init(done + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(summed + 8 * i, 1);
            bar_init(written + 8 * i, 2 * kWriteWarps);
        }
        bar_init(drained, 1);
        fence_barrier_init();
        prefetch_map(&map_dy);
        prefetch_map(&map_a);
        prefetch_map(&map_dw);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    follow_predecessor();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // the other CTA's barriers exist
    tmem_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        // A stage's codes come as soon as those before them have been converted, its rows of dy a stage later, when the products
        // of what was there are done.
        uint32_t n = 0, m = 0;   // stages of codes and of dy on their way
        int dy_column = 0, dy_row = 0;   // of stage m
        const bool leader = elect_one();
        bool ok = true;
        auto load_dy = [&] {
            const uint32_t slot = m % kGradStages, use = m / kGradStages, dst = stages + slot * kGradStageBytes, bar = loaded + 8 * slot;
            if (use > 0 && !__all_sync(0xffffffffu, bar_wait(done + 8 * slot, (use - 1) & 1, giveup))) return false;
            if (leader) {
                bar_expect(bar, kDyBytes);
                tma_load(dst, &map_dy, dy_column, dy_row, bar);
                tma_load(dst + kLineBytes, &map_dy, dy_column + 64, dy_row, bar);
            }
            __syncwarp();
            ++m;
            return true;
        };
        for (int64_t t = t_first; t < p.tiles && ok; t += t_step) {
            const GradTile x = grad_tile(p, t);
            const int n0 = x.n0 + kGradHalf * rank, k0 = x.k0 + kGradHalf * rank;
            const float* s = p.a_scales + min(k0 / 128, p.kb - 1);
            const int steps = grad_steps(x);
            for (int i = 0; i < steps && ok; ++i) {
                const uint32_t slot = n % kGradStages, use = n / kGradStages;
                if (use > 0) ok = __all_sync(0xffffffffu, bar_wait(taken + 8 * slot, (use - 1) & 1, giveup));
                if (n == kWithheldBlock || !ok) { ok = false; break; }
                const uint32_t bar = coded + 8 * slot;
                const int r = x.r0 + kGradRows * i;
                if (leader) {
                    bar_expect(bar, kCodeBytes);
                    tma_load(stages + slot * kGradStageBytes + kDyBytes + kValueBytes, &map_a, k0, r, bar);
                }
                __syncwarp();
                const uint32_t to = scales + 4 * (slot * kGradRows + lane);
                if (r + lane < x.r1) copy4(to, s + (int64_t)(r + lane) * p.kb);
                if (r + lane + 32 < x.r1) copy4(to + 128, s + (int64_t)(r + lane + 32) * p.kb);
                copies_arrive(bar);
                if (n++ > 0) ok = load_dy();
                dy_column = n0;
                dy_row = r;
            }
        }
        if (ok && n > 0) ok = load_dy();
        if (!ok || *giveup.flag) {   // its loads in flight, for which no other role may wait
            const long long t0 = clock64();
            for (uint32_t j = n < kGradStages ? 0 : n - kGradStages; j < n; ++j)
                bar_drain(coded + 8 * (j % kGradStages), (j / kGradStages) & 1, t0);
            for (uint32_t j = m < kGradStages ? 0 : m - kGradStages; j < m; ++j)
                bar_drain(loaded + 8 * (j % kGradStages), (j / kGradStages) & 1, t0);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t instruction = mma_instruction_across(FP16, kGradTile, kGradTile);
            const uint64_t a0 = mma_descriptor_across(stages, kLineBytes), b0 = mma_descriptor_across(stages + kDyBytes, kLineBytes);
            const bool leader = elect_one();
            uint32_t n = 0, tile = 0;   // stages and tiles with rows
            bool ok = true;
            for (int64_t t = t_first; t < p.tiles && ok; t += t_step) {
                const GradTile x = grad_tile(p, t);
                const int steps = uniform(grad_steps(x));
                if (steps == 0) continue;
                const uint32_t u = tile & 1, d = tmem + u * kGradTile;
                if (tile >= 2) ok = __all_sync(0xffffffffu, bar_wait<kPairTensor>(written + 8 * u, (tile / 2 - 1) & 1, giveup));
                for (int i = 0; i < steps && ok; ++i, ++n) {
                    const uint32_t slot = n % kGradStages;
                    ok = __all_sync(0xffffffffu, bar_wait<kPairShared>(ready + 8 * slot, (n / kGradStages) & 1, giveup));
                    if (!ok) break;
                    if (leader) {
                        tmem_fence_after();
                        const int k_steps = min(kGradRows, x.r1 - x.r0 - kGradRows * i + 15) / 16;
                        const uint32_t at = slot * (kGradStageBytes >> 4);
#pragma unroll
                        for (int j = 0; j < kGradRows / 16; ++j)
                            if (j < k_steps) mma_half_pair(d, a0 + at + 128 * j, b0 + at + 128 * j, instruction, i == 0 && j == 0);
                        mma_commit_pair(done + 8 * slot);
                        if (i + 1 == steps) mma_commit_pair(summed + 8 * u);
                    }
                    __syncwarp();
                }
                ++tile;
            }
            if (leader) mma_commit_pair(drained);
        }
        __syncwarp();
    } else if (warp < kFirstConverter) {
        uint32_t tile = 0;
        bool ok = true;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int part = (warp - kFirstWriter) / 4 * kGradHalf;
        const uint32_t buffer = outs + (warp - kFirstWriter) * kOutBytes;
        for (int64_t t = t_first; t < p.tiles && ok; t += t_step) {
            const GradTile x = grad_tile(p, t);
            const bool some = x.r1 > x.r0;
            const uint32_t u = tile & 1;
            if (some) {
                const long long limit = kWaitCycles + kStageCycles * grad_steps(x);
                ok = __all_sync(0xffffffffu, bar_wait(summed + 8 * u, (tile / 2) & 1, giveup, limit));
                if (!ok) break;
                tmem_fence_after();
            }
            const int row = x.n0 + kGradHalf * rank + (warp & 3) * 32;
#pragma unroll 1
            for (int c = part; c < part + kGradHalf && x.k0 + c < p.inner && row < p.columns; c += 32) {
                uint32_t r[32];
                if (some) {
                    tmem_load32(r, tmem + lanes + u * kGradTile + c);
                    tmem_wait(r);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
                write_sums<FP16>(p, &map_dw, buffer, r, x.k0 + c, row, x.g);
            }
            if (some) {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) bar_arrive(written + 8 * u);
                    else pair_arrive<kPairTensor>(peer_smem(written + 8 * u, 0));
                }
                ++tile;
            }
        }
        if (lane == 0) stores_wait();
        __syncwarp();
    } else {
        const int team = (warp - kFirstConverter) / kConvertTeam, thread = (int)(threadIdx.x - 32 * kFirstConverter) % (32 * kConvertTeam);
        const int row = thread / 8, piece = lane & 7;   // 16 codes of every (4 * kConvertTeam)th row from `row` on
        const uint32_t to0 = (uint32_t)(kDyBytes + piece / 4 * kLineBytes), other = piece / 4;
        const uint32_t first_ready = peer_smem(ready, 0);
        uint32_t n = 0;
        bool ok = true;
        for (int64_t t = t_first; t < p.tiles && ok; t += t_step) {
            const GradTile x = grad_tile(p, t);
            const int steps = grad_steps(x);
            for (int i = 0; i < steps; ++i, ++n) {
                const uint32_t slot = n % kGradStages, use = n / kGradStages;
                if (slot != (uint32_t)team) continue;
                const uint32_t stage = stages + slot * kGradStageBytes;
                ok = __all_sync(0xffffffffu, bar_wait(coded + 8 * slot, use & 1, giveup));
                if (!ok) break;
                const int left = x.r1 - x.r0 - kGradRows * i;   // rows of this stage that are the group's
                constexpr int kTimes = kGradRows / (4 * kConvertTeam);
                uint4 c[kTimes];
                float s[kTimes];
#pragma unroll
                for (int h = 0; h < kTimes; ++h) {
                    c[h] = smem_load4(stage + kDyBytes + kValueBytes + (row + 4 * kConvertTeam * h) * kGradHalf + 16 * piece);
                    s[h] = smem_load(scales + 4 * (slot * kGradRows + row + 4 * kConvertTeam * h));
                }
                if (use > 0) ok = __all_sync(0xffffffffu, bar_wait(done + 8 * slot, (use - 1) & 1, giveup));
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < kTimes; ++h) {
                    const int r = row + 4 * kConvertTeam * h;
                    // the lanes of the second line begin with their other half, so that each eight lanes, which hold a row,
                    // fill all banks with a store: both lines' rows lie on the same
                    const uint32_t word[4] = {other ? c[h].z : c[h].x, other ? c[h].w : c[h].y, other ? c[h].x : c[h].z,
                                              other ? c[h].y : c[h].w};
                    uint32_t v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 lo = mul2(e4m3x2_to_float2(word[j] & 0xFFFFu), both(s[h]));
                        const float2 hi = mul2(e4m3x2_to_float2(word[j] >> 16), both(s[h]));
                        v[2 * j] = r < left ? pack2<FP16>(lo.x, lo.y) : 0u;
                        v[2 * j + 1] = r < left ? pack2<FP16>(hi.x, hi.y) : 0u;
                    }
                    const uint32_t to = stage + to0 + r * 128, at = 2 * (piece & 3) + other, swap = r & 7;
                    smem_store4(to + ((at ^ swap) << 4), make_uint4(v[0], v[1], v[2], v[3]));
                    smem_store4(to + ((at ^ 1 ^ swap) << 4), make_uint4(v[4], v[5], v[6], v[7]));
                }
                // Behind the fence, because the next codes come by the asynchronous unit, which no barrier alone orders after this
                // warp's reads: handed back as soon as they were read, a stage in some million had the next one's codes.
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(taken + 8 * slot);
                ok = __all_sync(0xffffffffu, bar_wait(loaded + 8 * slot, use & 1, giveup));
                if (!ok) break;
                // the rest of the last 16 rows that are multiplied: dy's rows there are another group's
                if (left < kGradRows) {
                    const int q = thread & 15, end = (left + 15) / 16 * 16;
                    for (int r = left + thread / 16; r < end; r += 2 * kConvertTeam)
                        smem_store4(stage + q / 8 * kLineBytes + r * 128 + 16 * (q & 7), make_uint4(0, 0, 0, 0));
                    fence_async();
                }
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) bar_arrive(ready + 8 * slot);
                    else pair_arrive<kPairShared>(first_ready + 8 * slot);
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    // Tensor memory is freed, and the second CTA's barriers go, only after the last product has told both.  Here and not before,
    // so that the limit counts from the end of this CTA's other roles, however long the kernel's work takes.
    if (warp == 1 && elect_one()) bar_drain(drained, 0, clock64());
    cluster_sync();   // no product, arrival or read of the pair's memory is under way
    if (warp == 1) {
        tmem_fence_after();
        tmem_free_pair(tmem, 512);
    }
}

template <bool FP16>
cudaError_t launch_gradient(const GradArgs& p, const CUtensorMap& dy, const CUtensorMap& a, const CUtensorMap& dw, int sms,
                            cudaStream_t s)
{
    const cudaError_t e = allow_all_shared<ep_weight_gradient_kernel<FP16>>();
    if (e != cudaSuccess) return e;
    const int64_t pairs = p.tiles < sms / 2 ? p.tiles : sms / 2;
    return launch_cluster(ep_weight_gradient_kernel<FP16>, (unsigned)(2 * pairs), kGradThreads, kGradShared, 2, s, p, dy, a, dw);
}

}  // namespace
}  // namespace ep

extern "C" int ep_matmul_fp8_weight_gradient(const void* dy, int dtype, const void* a, const float* a_scales,
                                             const int32_t* offsets, int64_t rows, int groups, int columns, int inner,
                                             int out_fp32, void* dw, int32_t* device_status, void* stream)
{
    using namespace ep;
    const char* who = "ep_matmul_fp8_weight_gradient";
    if (rows < 0 || rows > INT32_MAX - kGradRows)
        return layer_fail(EP_ERR_ARG, "%s: rows=%lld outside 0..2^31-1-%d", who, (long long)rows, kGradRows);
    if (groups < 1 || groups > kMaxGradGroups || (!offsets && groups != 1))
        return layer_fail(EP_ERR_ARG, "%s: groups=%d outside 1..%d, or several without offsets", who, groups, kMaxGradGroups);
    if (inner < 16 || inner % 16 != 0 || inner > 1 << 20)
        return layer_fail(EP_ERR_ARG, "%s: inner=%d is not a multiple of 16 in 16..2^20", who, inner);
    if (columns < 8 || columns % 8 != 0 || columns > 1 << 20)
        return layer_fail(EP_ERR_ARG, "%s: columns=%d is not a multiple of 8 in 8..2^20", who, columns);
    if (dtype != EP_BF16 && dtype != EP_FP16)
        return layer_fail(EP_ERR_ARG, "%s: dtype=%d is neither EP_BF16 nor EP_FP16", who, dtype);
    if (!layer_aligned(device_status, 4))
        return layer_fail(EP_ERR_ARG, "%s: device_status is NULL or not 4-byte aligned", who);
    if (!layer_aligned(dw, 16)) return layer_fail(EP_ERR_ARG, "%s: dw is NULL or not 16-byte aligned", who);
    if (offsets && !layer_aligned(offsets, 4)) return layer_fail(EP_ERR_ARG, "%s: offsets is not 4-byte aligned", who);
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0)   // no row in any group
        return layer_cuda(cudaMemsetAsync(dw, 0, (size_t)groups * columns * inner * (out_fp32 ? 4 : 2), s), who);
    if (!layer_aligned(dy, 16) || !layer_aligned(a, 16) || !layer_aligned(a_scales, 4))
        return layer_fail(EP_ERR_ARG, "%s: dy, a or a_scales is NULL or misaligned", who);
    GradArgs p{};
    p.a_scales = a_scales; p.offsets = offsets; p.status = device_status; p.rows = rows; p.groups = groups;
    p.columns = columns; p.inner = inner; p.kb = (inner + 127) / 128;
    p.n_tiles = (columns + kGradTile - 1) / kGradTile; p.k_tiles = (inner + kGradTile - 1) / kGradTile;
    p.tiles = (int64_t)groups * p.n_tiles * p.k_tiles;
    p.out_fp32 = out_fp32 != 0;
    const int sms = layer_num_sms();
    if (sms < 2) return layer_fail(EP_ERR_CUDA, "%s: cannot tell the current device's multiprocessors", who);
    CUtensorMap m_dy, m_a, m_dw;
    const bool fp16 = dtype == EP_FP16;
    const CUtensorMapDataType half = fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (int rc = make_tile_map(&m_dy, who, "dy", dy, half, 2, rows, columns, kGradRows, 64, true)) return rc;
    if (int rc = make_tile_map(&m_a, who, "a", a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, inner, kGradRows, kGradHalf, false))
        return rc;
    const cuuint64_t size = p.out_fp32 ? 4 : 2, row_bytes = size * inner;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)columns, (cuuint64_t)groups}, pitch[2] = {row_bytes, row_bytes * columns};
    const cuuint32_t box[3] = {p.out_fp32 ? 16u : 32u, 32, 1};
    if (int rc = make_box_map(&m_dw, who, "dw", dw, p.out_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : half, 3, dims, pitch, box,
                              CU_TENSOR_MAP_SWIZZLE_64B))
        return rc;
    const cudaError_t e = fp16 ? launch_gradient<true>(p, m_dy, m_a, m_dw, sms, s) : launch_gradient<false>(p, m_dy, m_a, m_dw, sms, s);
    return layer_cuda(e, "ep_matmul_fp8_weight_gradient: launch");
}
