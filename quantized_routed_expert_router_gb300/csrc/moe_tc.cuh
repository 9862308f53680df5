// moe_tc.cuh - what the tensor-core products share (moe_fp8.cu, moe_matmul.cu):
// mbarriers with bounded waits, TMA and asynchronous copies, tcgen05, clusters.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {
namespace {

// bound on every device-side wait, in units of 2^16 SM clock cycles (8e8 cycles: under a second), unless a test
// hook shortens it; waits for copies and products in flight on the way out keep it
constexpr uint32_t kWaitLimit = 12207;

// position in the ring of stages
template <int N>
struct Ring {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ uint32_t sa(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sa(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %2, 0;\n @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(
            sa(b)), "r"(bytes), "r"(me)
        : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b, uint32_t me) {
    asm volatile("{\n .reg .pred e;\n setp.ne.u32 e, %1, 0;\n @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(sa(b)),
                 "r"(me)
                 : "memory");
}
// bits 16 .. 47 of the cycle counter
__device__ __forceinline__ uint32_t clock_hi() { return (uint32_t)((unsigned long long)clock64() >> 16); }
__device__ __forceinline__ bool bar_test(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(sa(b)), "r"(parity) : "memory");
    return ok != 0;
}
// Barriers at which another block of the cluster arrives, or its tensor cores do: the wait acquires, and the arrival releases,
// at the cluster's scope, by fences that are about shared memory alone.  With mbarrier's own .release.cluster and
// .acquire.cluster, which are about all memory, a stage's hand-over between two blocks took 2000 cycles (8192^3: 1757 us, so
// 597); with the release alone on the hand-over of TMEM buffers fp32 results waited for the epilogue's stores (8192 x 2048 by
// 7168 x 2048: 195 us, so 174).
__device__ __forceinline__ bool bar_test_cluster(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n"
        " @p fence.acquire.sync_restrict::shared::cluster.cluster;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(sa(b)), "r"(parity) : "memory");
    return ok != 0;
}
// arrives at the barrier at the same place in block `rank` of the cluster
__device__ __forceinline__ void bar_arrive_at(uint64_t *b, uint32_t rank, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 at;\n setp.ne.u32 e, %2, 0;\n mapa.shared::cluster.u32 at, %0, %1;\n"
        " @e fence.release.sync_restrict::shared::cta.cluster;\n"
        " @e mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [at];\n}" ::"r"(sa(b)), "r"(rank), "r"(me)
        : "memory");
}
// 1 in one lane of a converged warp.  The single-thread instructions (copies,
// products, commits, arrivals) are predicated on it in straight code that the
// whole warp runs: a branch around them costs more than they do (a stage of
// products took 540 cycles to issue behind a test of the lane number, 260 behind
// a branch on this, 200 predicated).
__device__ __forceinline__ uint32_t elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p;
}
// wait for a phase; false once this block has given up (the first wait to run
// out says so to the others, in *abort in shared memory, and in the status word).
// CLUSTER: another block, or its tensor cores, arrive at the barrier.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, int *abort, uint32_t limit, unsigned *status) {
    const auto test = [&] { return CLUSTER ? bar_test_cluster(b, parity) : bar_test(b, parity); };
    if (test()) return true;
    const uint32_t t0 = clock_hi();
    while (!test()) {
        if (*(volatile int *)abort) return false;
        if (clock_hi() - t0 > limit) {
            *(volatile int *)abort = 1;
            atomicOr(status, MOE_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}
// wait on the way out of a block: for its own copies and products in flight,
// until kWaitLimit after t0 at most
__device__ __forceinline__ void bar_settle(uint64_t *b, uint32_t parity, uint32_t t0) {
    while (!bar_test(b, parity))
        if (clock_hi() - t0 > kWaitLimit) return;
}
__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *m, int x, int y, uint64_t *bar, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %5, 0;\n"
        " @e cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(
            sa(dst)), "l"(m), "r"(x), "r"(y), "r"(sa(bar)), "r"(me)
        : "memory");
}
// 16 bytes, or 16 zeros where `bytes` is 0
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// shared-memory descriptor of a K-major tile with 128-byte rows and the
// 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_commit(uint64_t *bar, uint32_t me) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.u32 e, %1, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(sa(bar)), "r"(me)
        : "memory");
}
// 32 columns of TMEM into registers.  A load is asynchronous: its registers hold the values only once the thread has waited
// for it, and what follows has to say so to the compiler, which moves arithmetic past statements that do not name its operands
// (a "memory" clobber does not hold it).  So the values come out of the statement that waits: load and wait are one, or a load
// that has other work behind it hands its registers to tmem_landed.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32_begin(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
// waits for this thread's loads, those into v among them
__device__ __forceinline__ void tmem_landed(uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
          "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
          "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
          "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
        :
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 ld_peer(uint32_t addr, uint32_t rank) {
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float ld_peer1(uint32_t addr, uint32_t rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

}  // namespace
}  // namespace moe
