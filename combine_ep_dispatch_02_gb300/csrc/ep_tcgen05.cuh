// ep_tcgen05.cuh -- the asynchronous machinery the product kernels use, as inline PTX: mbarriers with
// bounded waits, tiled TMA loads, and the fifth-generation tensor cores with their tensor memory.
//
// Bounded waits.  Every wait gives up after kWaitCycles clock cycles (or as soon as another thread of
// the CTA gave up), records EP_ERR_DEVICE_TIMEOUT and returns false.  The warps that load and those that
// make factors then leave; the multiplying and the scaling warps go through all their blocks, on whatever
// is there, because named barriers, whose waits have no limit, need every warp's arrivals in step.  What
// is in flight is waited for (bounded again), tensor memory is freed, and the kernel returns.
#pragma once

#include <cuda.h>

#include "ep_layer.cuh"

namespace ep {

// a second and a half at 2 GHz; the longest legitimate wait is a tile's, under a millisecond
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

// Wait until the barrier's phase of this parity has completed; false if the wait gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Giveup& g)
{
    if (bar_test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
        if (*g.flag) return false;
        if (clock64() - t0 > kWaitCycles) {
            *g.flag = 1;
            record_status(g.status, EP_ERR_DEVICE_TIMEOUT);
            return false;
        }
    }
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

#endif  // __CUDACC__

}  // namespace ep
