// situ_pair.cuh — what the linear operator's tensor-core kernels share: products on a PAIR of SMs
// (tcgen05 cta_group::2).
//
// The two CTAs of a cluster of 2 work on one 256-row tile: each holds its own 128 rows of A, half of B's
// rows, and 128 rows of the accumulator, and one thread of the leader (cluster rank 0) issues the MMAs
// of both. Each SM then loads and keeps half of a 256-wide B tile instead of all of it: 32 KB a 64-deep
// stage instead of 48 KB for the same products.
//
// Barriers (all in each CTA's shared memory, at the same offsets):
//   full[s]    leader's: the loads of both CTAs into stage s count there (transaction bytes of both)
//   empty[s]   both: the leader's commit of the MMAs that read stage s arrives at both
//   tfull[a]   both: the commit of the MMAs into accumulator a
//   tempty[a]  leader's: every epilogue warp of both CTAs, when it has read its part of a
// Every mbarrier wait is bounded as in situ_tc.cuh. TMEM: one CTA per SM and the same 512 columns in both,
// allocated and freed by warp 1 of both; the cluster barriers at the start and end keep either CTA from
// touching the other's barriers or memory before they are set up or after it has left.
#pragma once

#include "situ_tc.cuh"

namespace situ_pair {

using namespace situ_tc;

constexpr int PSTAGES = 8;                   // most stages of a ring (barriers); a kernel may use fewer, larger ones
constexpr int PA_BYTES = 128 * BK * 2;       // this CTA's 128 rows of A (or columns, MN-major)
constexpr int PB_BYTES = 128 * BK * 2;       // this CTA's half of 256 rows of B (or columns)
constexpr int PRING_BYTES = 196 * 1024;     // 6 stages for 256 rows of B, 7 for 192, 8 for 128
constexpr int PBOX_BYTES = 64 * BK * 2;      // an MN-major box: 64 columns x 64 deep

struct alignas(8) PairBars {
    uint64_t full[PSTAGES];
    uint64_t empty[PSTAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t tail_full[PSTAGES];             // weight gradient: this CTA's loads of an expert's last, ragged stage
    uint64_t tail_ready[PSTAGES];            // leader's: both CTAs have zeroed the rows past the expert's end in it
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
};

// One poll: the thread is suspended until the phase completes or about SUSPEND_NS have passed.
constexpr uint32_t SUSPEND_NS = 20000;
__device__ __forceinline__ bool try_wait_cluster(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(b)), "r"(parity), "r"(SUSPEND_NS)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool try_wait_cta(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_addr(b)), "r"(parity), "r"(SUSPEND_NS)
        : "memory");
    return ok != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// Bounded wait of a converged warp (2 s by %globaltimer, or POLL_LIMIT polls): on a timeout sets the CTA's abort flag and the
// caller's status word; returns false then, and once another role of the CTA has aborted, to all lanes alike.
// CLUSTER: acquire at cluster scope, for barriers at which threads of the other CTA arrive.
//
// The roles that wait here feed the tensor cores, so what surrounds a wait counts: a pair's 64-deep block takes 512
// cycles, some 90 dependent instructions of one thread. Hence the suspended try_wait (hot polls of the waiting
// warps slowed the issuing ones: 19456 x 3584 x 3584 in 378 us instead of 309), the clock (several hundred ns to
// read) only after FREE_POLLS polls, and votes, which keep control flow and so descriptors and
// coordinates uniform over the warp: in a single-lane branch each MMA and load first moved six values to
// uniform registers.
constexpr uint32_t FREE_POLLS = 16;
constexpr uint32_t POLL_LIMIT = 1u << 19;    // of at most 20 us: some ten seconds

template <bool CLUSTER = false>
__device__ __forceinline__ bool pair_wait(uint64_t* b, uint32_t parity, int* abort, int* status) {
    for (uint32_t i = 0; i < FREE_POLLS; ++i)
        if (__all_sync(0xffffffffu, CLUSTER ? try_wait_cluster(b, parity) : try_wait_cta(b, parity))) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < POLL_LIMIT; ++i) {
        if (__all_sync(0xffffffffu, CLUSTER ? try_wait_cluster(b, parity) : try_wait_cta(b, parity))) return true;
        if ((i & 63) == 63) {
            if (__any_sync(0xffffffffu, *(volatile int*)abort)) return false;
            if (__any_sync(0xffffffffu, global_ns() - t0 > WAIT_NS)) break;
        }
    }
    *(volatile int*)abort = 1;
    if (status) atomicExch(status, 1);
    return false;
}

// All epilogue warps (2 .. epi_warps + 1): wait for a finished accumulator. Only warp 2 polls; the others wait at a
// named barrier, which takes no issue slots. The result is the same over a warp.
__device__ __forceinline__ bool pair_wait_epilogue(uint64_t* b, uint32_t parity, PairBars* bars, int* status,
                                                   int epi_warps) {
    if ((threadIdx.x >> 5) == 2 && !*(volatile int*)&bars->abort) pair_wait(b, parity, &bars->abort, status);
    epi_barrier(epi_warps * 32);
    const bool ok = __all_sync(0xffffffffu, !*(volatile int*)&bars->abort);   // tcgen05.ld is warp-collective
    tc_fence_after();
    return ok;
}

// Box loads into this CTA's shared memory whose bytes count at `bar`, a shared::cluster address: the
// leader's barrier, from either CTA of the pair (that is what .cta_group::2 allows).
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

// Instruction descriptor, kind::f16 on a pair: fp32 accumulate, bf16 operands, M = 256, N columns
// (a multiple of 32 up to 256); bits 15 / 16: A / B stored MN-major.
__device__ __forceinline__ uint32_t pair_idesc(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
}

__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// When the MMAs issued so far are done: one arrival at this barrier of both CTAs.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// All threads of both CTAs: barriers, TMEM (512 columns), cluster barrier. epi_warps: epilogue warps per CTA.
__device__ __forceinline__ uint32_t pair_setup(PairBars* bars, int epi_warps) {
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < PSTAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
            mbar_init(&bars->tail_full[s], 1);
            mbar_init(&bars->tail_ready[s], 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&bars->tfull[a], 1);
            mbar_init(&bars->tempty[a], (uint32_t)(2 * epi_warps));
        }
        mbar_init(&bars->mma_done, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&bars->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    return bars->tmem_base;
}

// All threads of both CTAs, when every role is done (the leader's MMA warp has committed to mma_done last): its
// arrivals at this CTA's barriers are in before either CTA leaves.
__device__ __forceinline__ void pair_teardown(uint32_t tmem, PairBars* bars) {
    tc_fence_before();
    __syncthreads();
    if ((threadIdx.x >> 5) == 1) mbar_drain(&bars->mma_done, 0);
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if ((threadIdx.x >> 5) == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
}

// The leader's producer at the end (normal or aborted): the loads of both CTAs that were counted at its full
// barriers have landed, or two seconds have passed. In a finished run every stage's last phase is complete and
// this costs nothing; after an abort a phase whose other half was never issued runs into the limit.
__device__ __forceinline__ void pair_drain(PairBars* bars, uint32_t pending, uint32_t parity) {
    for (int s = 0; s < PSTAGES; ++s)
        if (pending & (1u << s)) mbar_drain(&bars->full[s], (parity >> s) & 1u);
}

// Launch as clusters of 2, one CTA per SM, at most `pairs` clusters.
template <class... KArgs, class... Args>
inline cudaError_t launch_pairs(void (*kernel)(KArgs...), int64_t pairs, int threads, int smem, cudaStream_t stream,
                                Args... args) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (pairs > sms / 2) pairs = sms / 2;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace situ_pair
