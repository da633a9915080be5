// ep_tcgen05.cuh -- the asynchronous machinery the product kernels use, as inline PTX: mbarriers with
// bounded waits, tiled TMA loads, and the fifth-generation tensor cores with their tensor memory.
//
// Bounded waits.  Every wait gives up after kWaitCycles clock cycles, or the longer limit that a wait for a whole tile is
// given (or as soon as another thread of the CTA gave up), records EP_ERR_DEVICE_TIMEOUT and returns false.  The warps that
// load and those that make factors then leave; the multiplying and the scaling warps go through all their blocks, on whatever
// is there, because named barriers, whose waits have no limit, need every warp's arrivals in step.  What
// is in flight is waited for (bounded again), tensor memory is freed, and the kernel returns.
#pragma once

#include <cuda.h>

#include "ep_layer.cuh"

namespace ep {

// a second and a half at 2 GHz; the longest legitimate wait of this limit is that of a product's tile, whose K of 2^20
// at the most is 8192 blocks of some 1000 cycles, 4 ms
#ifndef EP_WAIT_CYCLES
#define EP_WAIT_CYCLES (3ll << 30)
#endif
constexpr long long kWaitCycles = EP_WAIT_CYCLES;

// Test builds (EP_TEST_WITHHOLD_LOAD): block 2 of every loading warp is never loaded, so that the waits
// for it run out.
#ifdef EP_TEST_WITHHOLD_LOAD
constexpr uint32_t kWithheldBlock = 2;
#else
constexpr uint32_t kWithheldBlock = ~0u;
#endif

// a thread that waits sleeps for up to this long before it looks again: polling slows the barriers down
constexpr uint32_t kSuspendNs = 1000000;

#ifdef __CUDACC__

// One lane of a converged warp, in a form the compiler knows to be one lane.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
    return e != 0;
}

// A value that is the same in every lane, told to the compiler: descriptors and loop counts made from it
// stay in uniform registers, which the tensor-core instructions read.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ float smem_load(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void smem_store4(uint32_t addr, const float2& lo, const float2& hi)
{
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "f"(lo.x), "f"(lo.y), "f"(hi.x), "f"(hi.y) : "memory");
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(kSuspendNs) : "memory");
    return ok != 0;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// The CTA's shared flag that a wait has given up, and the caller's status word.
struct Giveup {
    volatile int* flag;
    int* status;
};

// Whose arrivals a barrier takes, and so what a wait for its phase orders: this CTA's threads and asynchronous units; or both
// CTAs' of a pair (pair_arrive below), which leaves tensor memory to the caller's tmem_fence_after(), or orders what both wrote
// to their shared memory too.
enum Arrivals { kOwnArrivals, kPairTensor, kPairShared };

template <Arrivals FROM>
__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity, bool wait)
{
    if constexpr (FROM == kOwnArrivals) return wait ? bar_try(bar, parity) : bar_test(bar, parity);
    uint32_t ok;
    if (wait)
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(bar), "r"(parity), "r"(kSuspendNs) : "memory");
    else
        asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// Wait until the barrier's phase of this parity has completed; false if the wait gave up.
template <Arrivals FROM = kOwnArrivals>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Giveup& g, long long limit = kWaitCycles)
{
    if (!bar_done<FROM>(bar, parity, false)) {
        const long long t0 = clock64();
        while (!bar_done<FROM>(bar, parity, true)) {
            if (*g.flag) return false;
            if (clock64() - t0 > limit) {
                *g.flag = 1;
                record_status(g.status, EP_ERR_DEVICE_TIMEOUT);
                return false;
            }
        }
    }
    if constexpr (FROM == kPairShared) asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
    return true;
}

// A scaling warp's wait for a block's products, by a whole warp.  The multiplying warp issues every block,
// the latest when its own wait for the loads has given up, so this one does not end when another gave
// up: a scaling warp that ran ahead would arrive twice where the others arrive once, and the multiplying
// warp could wait at its named barrier for ever.  The limit is that of a tensor core that has stopped.
__device__ __forceinline__ void products_wait(uint32_t bar, uint32_t parity, const Giveup& g)
{
    if (!bar_test(bar, parity)) {
        const long long t0 = clock64();
        while (!bar_try(bar, parity)) {
            if (clock64() - t0 > 8 * kWaitCycles) {
                *g.flag = 1;
                record_status(g.status, EP_ERR_DEVICE_TIMEOUT);
                break;
            }
        }
    }
    __syncwarp();
}

// The wait of a role that is leaving early for its own operations in flight, since t0: bounded, records nothing.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity, long long t0)
{
    while (!bar_try(bar, parity) && clock64() - t0 < kWaitCycles) {}
}

// ---- between the CTAs of a cluster

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// The address in CTA `rank` of the cluster that corresponds to this CTA's shared-memory address.
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float peer_load(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 peer_load4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Arrive on a peer's barrier; this thread's earlier writes, and those ordered before them, are visible to
// whoever waits for the phase with peer_wait().
__device__ __forceinline__ void peer_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ bool peer_wait(uint32_t bar, uint32_t parity, const Giveup& g)
{
    const bool ok = bar_wait(bar, parity, g);
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    return ok;
}

// No CTA of the cluster leaves while another may still reach its shared memory.
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Barrier initialisations become visible to the asynchronous units.
__device__ __forceinline__ void fence_barrier_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m)
{
    asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory");
}

// Box of a 2-D tensor map at (x, y) into shared memory; x is a multiple of 16 bytes in every call.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}

// ---- tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns)   // one warp
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns)    // the same warp
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(columns));
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive columns of this warp's 32 lanes: lane i gets row i's.  Complete after tmem_wait().
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

// 16 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

// The registers are tied to the wait, so that no use of them can be scheduled before it.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// d += a * b for two floats each, one instruction: rounded as two fused multiply-adds.  Kept in the
// order it is written in, between the loads that it is meant to overlap.
__device__ __forceinline__ void fma2(float2& d, const float2& a, const float2& b)
{
    asm volatile("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%0, %1};\n\t"
        "fma.rn.f32x2 z, x, y, z; mov.b64 {%0, %1}, z; }"
        : "+f"(d.x), "+f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

// ---- matrix multiply-accumulate

// Shared-memory descriptor of a K-major operand whose rows are 128 bytes, swizzled by 128 bytes:
// groups of 8 rows are 1024 bytes apart.  The tile starts on a 1024-byte boundary; stepping 32 bytes
// along K adds 32 to the address.
__device__ __forceinline__ uint64_t mma_descriptor(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// Instruction descriptor: FP32 accumulator, e4m3 A and B, both K-major, M x N.
__host__ __device__ constexpr uint32_t mma_instruction(int m, int n)
{
    return 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// D (tensor memory) = A B^T over 32 elements of K, plus D unless first.  One thread.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, bool first)
{
    asm volatile("{ .reg .pred p; setp.eq.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
                 :: "r"(d), "l"(a), "l"(b), "r"(instruction), "r"((uint32_t)first) : "memory");
}

// Arrive on the barrier when every product issued so far by this thread has finished.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}

// ---- the same by a pair of CTAs (a cluster of two), each holding half of the rows of A and of D and half of B's columns
//
// Both CTAs allocate and free; the products are issued by one thread of the first, with the addresses that the operands
// have in its own shared memory, which are those in the second's too.

__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot, uint32_t columns)   // one warp of each CTA
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_pair(uint32_t base, uint32_t columns)    // the same warps
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(columns));
}

// Shared-memory descriptor of a 16-bit operand that lies along its rows or columns rather than along K: K lines of 64
// elements, 128 bytes each, swizzled by 128 bytes; groups of 8 lines 1024 bytes apart, the next 64 elements `next` bytes
// further on.  Stepping 16 along K adds 2048 to the address.
__device__ __forceinline__ uint64_t mma_descriptor_across(uint32_t addr, uint32_t next)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(next >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// Instruction descriptor: FP32 accumulator, BF16 or FP16 A and B, both across K, M x N.
__host__ __device__ constexpr uint32_t mma_instruction_across(bool fp16, int m, int n)
{
    return 1u << 4 | (fp16 ? 0u : 1u << 7 | 1u << 10) | 1u << 15 | 1u << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// D = A B over 16 elements of K, plus D unless first.  One thread of the first CTA.
__device__ __forceinline__ void mma_half_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, bool first)
{
    asm volatile("{ .reg .pred p; setp.eq.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }"
                 :: "r"(d), "l"(a), "l"(b), "r"(instruction), "r"((uint32_t)first) : "memory");
}

// Arrive on both CTAs' barriers at this address when every product issued so far by this thread has finished.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"((uint16_t)3) : "memory");
}

// The second CTA's arrival on a barrier of the pair's first, whose waits are of the same kind.  kPairTensor: the thread's use of
// tensor memory before tmem_fence_before() is over.  kPairShared: this CTA's shared memory, written before fence_async(), may be
// multiplied.  The fence is held to shared memory: one of everything, an arrival with release semantics for the cluster, takes a
// thousand cycles longer (8192 rows in 8 groups of 4096 x 7168 377 us; 319 so; 314 ordered within the CTA alone, which the
// memory model does not carry to the other CTA's thread that issues the products).
template <Arrivals TO>
__device__ __forceinline__ void pair_arrive(uint32_t bar)
{
    static_assert(TO != kOwnArrivals, "bar_arrive");
    if constexpr (TO == kPairShared) asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

// This thread's writes to shared memory become visible to the asynchronous units.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Four bytes of global memory into shared memory, asynchronously, and this thread's arrival on a barrier when its copies
// so far have landed (the barrier counts that arrival).
__device__ __forceinline__ void copy4(uint32_t to, const void* from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(bar) : "memory");
}

// A box of shared memory to global memory, asynchronously, by one thread; the thread's stores are one group each, and
// stores_wait_read() returns when their bytes have been read, stores_wait() when they have been written.
__device__ __forceinline__ void tma_store3(const CUtensorMap* map, uint32_t from, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :: "l"(map), "r"(from), "r"(x), "r"(y), "r"(z) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint4 smem_load4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void smem_store4(uint32_t addr, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 64 consecutive columns, n of which exist, of a warp's 32 rows, m of which exist (row by lane, rows `pitch` bytes
// apart), 16-bit: w holds a lane's row in 32-byte pieces.  A store of 32 bytes by every lane to a row of its own visits 32
// lines, two cycles each, 4000 for a tile.  So four lanes first trade the pieces, two exchanges of half of
// them, until lane q of the four holds piece q of all four rows: a store then writes 128 bytes each of 8 rows.
__device__ __forceinline__ void store_lines(uint8_t* out, int64_t pitch, uint32_t (&w)[4][8], int m, int n, int vec)
{
    const int lane = threadIdx.x & 31, q = lane & 3;
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
    const int left = n - 16 * q;   // columns of this lane's pieces that exist
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = (lane & ~3) + r;
        if (row >= m) break;
        uint8_t* to = out + row * pitch + 32 * q;
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

// The same for 2 * PAIRS columns that are still FP32.
template <bool FP16, int PAIRS>
__device__ __forceinline__ void store_rows(uint8_t* out, int64_t pitch, const float2 (&acc)[PAIRS], int m, int n, int vec)
{
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
        store_lines(out + 128 * h, pitch, w, m, n - 64 * h, vec);
    }
}

// ---- host side: tensor maps and cluster launches

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled()
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

// Map of a dense array of `rank` dimensions, innermost first, with boxes of `box`; elements past an end read as zeros and are
// not written.
inline int make_box_map(CUtensorMap* m, const char* who, const char* what, const void* base, CUtensorMapDataType type, int rank,
                        const cuuint64_t* dims, const cuuint64_t* pitch, const cuuint32_t* box, CUtensorMapSwizzle swizzle)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return layer_fail(EP_ERR_CUDA, "%s: the driver has no cuTensorMapEncodeTiled", who);
    const cuuint32_t step[3] = {1, 1, 1};
    auto make = [&] {
        return encode(m, type, rank, const_cast<void*>(base), dims, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = make();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {   // a host thread's first call, which nothing has bound to the device yet
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaSetDevice(dev);
        if (e != cudaSuccess) {
            layer_cuda(e, who);
            return layer_fail(EP_ERR_CUDA, "%s: binding the host thread to its device: %s", who, cudaGetErrorString(e));
        }
        r = make();
    }
    if (r != CUDA_SUCCESS) return layer_fail(EP_ERR_CUDA, "%s: tensor map of %s: CUresult %d", who, what, (int)r);
    return EP_OK;
}

// Of [rows][columns], elements of `size` bytes, with boxes of box_rows x box_columns, swizzled by 128 bytes or not at all.
inline int make_tile_map(CUtensorMap* m, const char* who, const char* what, const void* base, CUtensorMapDataType type, int size,
                         int64_t rows, int64_t columns, int box_rows, int box_columns, bool swizzled)
{
    const cuuint64_t dims[2] = {(cuuint64_t)columns, (cuuint64_t)rows}, pitch[1] = {(cuuint64_t)columns * size};
    const cuuint32_t box[2] = {(cuuint32_t)box_columns, (cuuint32_t)box_rows};
    return make_box_map(m, who, what, base, type, 2, dims, pitch, box, swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
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

#endif  // __CUDACC__

}  // namespace ep
