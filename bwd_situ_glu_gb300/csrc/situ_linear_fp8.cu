// situ_linear_fp8.cu — matrix product of quantised rows with their expert's (or the one dense) quantised weight, with bias,
// activation and residual in the epilogue, and the input gradient (include/situ_fp8.h).
//
//   forward   out[r] = act(Σ_kb 2^(ea[r,kb] + ew[·,kb]) Σ_{k in kb} a[r,k]·W_e[·,k] + b_e) + residual[r]
//   dgrad     da[r]  = the same over blocks of dz[r] and W_eᵀ
//
// As the bf16 product (situ_linear.cu): pairs of SMs, the weights as the MMA's 256-row operand, the rows as its N operand.
// What differs:
//   * tcgen05.mma kind::mxf8f6f4 with block scales: the tensor core multiplies each 32-deep step of a row by a
//     power of two held as a byte in TMEM, so the scales of 128-deep blocks cost neither instructions in the epilogue
//     nor a rounding. Two more warps of each CTA write the bytes of four blocks at a time (its 128 weight rows': one byte for
//     all; the chunk's rows': one each) in the layout that tcgen05.cp takes; the MMA warp copies them to TMEM in front of
//     the blocks' MMAs. Each byte stands four times in a word, once for each MMA of its block.
//     The hand-over (fetch, shared memory, proxy fence, arrival at the leader) is what the speed hung on, 16385 x 3584 x 3584:
//     block by block 380 us, four blocks at a time 168, the bytes fetched a turn ahead 160, two warps in turn 141, a group's copies
//     at its start, so that its buffer is free again a group earlier, 133. By %clock a block of 224 rows now takes 523 cycles,
//     jobs' ends included, 448 of them its products (of 168 rows of ragged experts, weights from HBM: 615 of 336). What is
//     left is power: the SMs run at 1.6 to 1.7 GHz in calls back to back, at 1.52 (1360 W) in a long run: 16384 rows 150 us,
//     2.8 PFLOP/s.
//   * two accumulators and the scales share TMEM's 512 columns, so a chunk has at most 224 rows.
//   * the dgrad reads W_e as stored (contraction apart, "MN-major"): boxes of 128 columns x 128 rows of bytes.
//   * linear_fp8_few_kernel: for few rows per expert, as there.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/situ_fp8.h"
#include "situ_device.cuh"
#include "situ_fp8.cuh"
#include "situ_host.h"
#include "situ_linear.cuh"
#include "situ_linear_tc.cuh"
#include "situ_pair.cuh"

namespace {

using namespace situ;
using namespace situ_host;
using namespace situ_pair;
using namespace situ_linear;
using namespace situ_linear_tc;
using namespace situ_fp8;

constexpr int KB8 = 128;                     // elements (bytes) of a block of the contraction: one scale
constexpr int UK8 = 32;                      // elements per tcgen05.mma
constexpr int MAX_CHUNK = 224;               // rows per job
constexpr int ACC_COLS = 224;                // TMEM columns of an accumulator
constexpr int SCALE_WARP = 2 + NUM_EPI_WARPS, SCALE_WARPS = 2;
constexpr int NUM_THREADS = (SCALE_WARP + SCALE_WARPS) * 32;    // TMA, MMA, epilogue, scales

// Scale bytes of a stage in shared memory: 128 rows are 512 bytes, row i at 16·(i % 32) + 4·(i / 32), as tcgen05.cp
// 32x128b takes them. One such piece for the weights, two for the rows.
constexpr int SCALE_PIECE = 512;
constexpr int SCALE_BYTES = 3 * SCALE_PIECE;
constexpr int SCALE_COL0 = 2 * ACC_COLS;     // in TMEM: 4 columns a piece
constexpr int GROUP_KB = 4, GROUPS = SCALE_WARPS;   // blocks whose scales are handed over at once; such groups in shared memory
// TMEM holds the scales of GROUP_KB blocks; the tensor core takes copies and MMAs of one thread in order
static_assert(SCALE_COL0 + GROUP_KB * 12 <= TMEM_COLS, "TMEM columns");

// A ring stage: two blocks, of each 128 weight rows and half of the chunk's rows, 128 bytes each. (Calls back to back, in stages of one
// block and of two, the ring's bytes the same: 448 rows over 112 experts of 3584 x 2048 135 / 129 us, 32768 rows 240 / 236; 4096 rows over
// 64 experts of 3584 x 3584 136 / 135, 16385 dense rows 130 / 131.)
constexpr int STAGE_KB = 2;
__host__ __device__ constexpr int block_bytes(int most) { return PA_BYTES + most / 2 * KB8; }
constexpr int RING_BYTES = 3 * STAGE_KB * block_bytes(MAX_CHUNK);
__host__ __device__ constexpr int ring_stages(int most) {
    const int s = RING_BYTES / (STAGE_KB * block_bytes(most));
    return s < PSTAGES ? s : PSTAGES;
}

struct alignas(8) ScaleBars {
    uint64_t full[GROUPS];                   // leader's: both CTAs have written a group
    uint64_t empty[GROUPS];                  // both: the commit of the MMAs behind a group's copies
    int rows[GROUPS];                        // leader's: the MMA's N of a group's job
};

constexpr int SMEM_BYTES = 1024 + RING_BYTES + GROUPS * GROUP_KB * SCALE_BYTES + NUM_EPI_WARPS * PATCH + (int)sizeof(PairBars) + (int)sizeof(ScaleBars) +
                           (int)sizeof(Plan);
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

// Instruction descriptor, kind::mxf8f6f4 on a pair: fp32 accumulate, E4M3 operands (formats 0), E8M0 scales (bit 23), scale
// bytes 0 of their words, M = 256, N columns (a multiple of 32); bit 15: A stored MN-major.
__device__ __forceinline__ uint32_t scaled_idesc(int n, bool a_mn) {
    return ((uint32_t)a_mn << 15) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(256 >> 7) << 27);
}

__device__ __forceinline__ void scaled_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa_tmem,
                                           uint32_t sb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of a piece of scales: no swizzle, 8 rows of 16 bytes are 128 bytes on.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// A piece to four TMEM columns of all four lane quadrants, in both CTAs (each from its own shared memory).
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// An MN-major tile of 128 columns (bytes) x 128 deep, as a TMA box writes it: a row of the contraction is 128 bytes, eight
// are a 1024-byte swizzle atom (stride byte offset); there is no second 128 columns (leading byte offset unused).
// The same fields as a K-major tile's.
__device__ __forceinline__ uint64_t smem_desc_mn8(uint32_t saddr) { return smem_desc(saddr); }

__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return a | (b << 8) | (c << 16) | (d << 24);
}

// A CTA's half of a chunk's rows is a multiple of 16: a map, and so one load a stage, for each (boxes of 16 (i + 1) rows).
constexpr int ROW_MAPS = MAX_CHUNK / 32;
struct RowMaps {
    CUtensorMap m[ROW_MAPS];
};

// Where a weight's scale bytes are: expert e's block of output columns c and block kb of the contraction at
// e·per_expert + c·col_step + kb·k_step.
struct ScaleStrides {
    int64_t per_expert;
    int col_step, k_step, col_blocks;
};

template <bool W_MN, int ACT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    linear_fp8_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_r,
                         const uint8_t* __restrict__ row_scales, const uint8_t* __restrict__ w_scales, ScaleStrides ws,
                         const int64_t* __restrict__ offsets, const float* __restrict__ bias,
                         const uint16_t* __restrict__ residual, void* __restrict__ out, int out_fp32,
                         uint16_t* __restrict__ pre, int* __restrict__ status, int E, int64_t R, int64_t NCOL, int KB,
                         int most) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* scales = ring + RING_BYTES;
    uint8_t* patches = scales + GROUPS * GROUP_KB * SCALE_BYTES;
    PairBars* bars = (PairBars*)(patches + NUM_EPI_WARPS * PATCH);
    ScaleBars* sbars = (ScaleBars*)(bars + 1);
    Plan& plan = *(Plan*)(sbars + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int NT = (int)((NCOL + TILE - 1) / TILE);
    const int bbytes = block_bytes(most), sbytes = STAGE_KB * bbytes, stages = ring_stages(most);

    if (threadIdx.x == 0) {                  // before pair_setup's fence and barriers
        for (int g = 0; g < GROUPS; ++g) {
            mbar_init(&sbars->full[g], 2);
            mbar_init(&sbars->empty[g], 1);
        }
    }
    const uint32_t tmem = pair_setup(bars, NUM_EPI_WARPS);
    dependents_wait();
    build_plan(plan, offsets, E, R, most);
    __syncthreads();
    const int jobs = plan.start[E] * NT;
    const int j0 = blockIdx.x >> 1, jstep = gridDim.x >> 1;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs; the warp converged, one lane issues)
        const bool elected = elect_one();
        int stage = 0;
        uint32_t phase = 0, pending = 0, pend_par = 0;
        const uint64_t pol_w = make_policy<kHintB>(), pol_r = make_policy<kHintA>();
        const uint32_t full0 = cluster_addr(&bars->full[0], 0);
        bool ok = true;
        Job next = {};
        if (j0 < jobs) next = job_at(j0, plan, E, NT);
        for (int j = j0; ok && j < jobs; j += jstep) {
            const Job q = next;
            const int c0 = q.nt * TILE + rank * 128, r0 = q.row0 + rank * (q.n >> 1);
            const uint32_t bytes = (uint32_t)(2 * PA_BYTES + q.n * KB8);
            const CUtensorMap* map_rows = &map_r.m[(q.n >> 5) - 1];
            for (int kb = 0; kb < KB; kb += STAGE_KB) {
                if (!pair_wait(&bars->empty[stage], phase ^ 1, &bars->abort, status)) { ok = false; break; }
                if (elected) {
                    const int blocks = min(STAGE_KB, KB - kb);
                    if (rank == 0) mbar_expect_tx(&bars->full[stage], bytes * blocks);
                    const uint32_t bar = full0 + (uint32_t)(stage * sizeof(uint64_t));
                    uint8_t* sa = ring + stage * sbytes;
#pragma unroll
                    for (int i = 0; i < STAGE_KB; ++i) {
                        if (i >= blocks) break;
                        const int k = (kb + i) * KB8;
                        if constexpr (W_MN) pair_load_3d(sa + i * bbytes, &map_w, c0, k, q.e, bar, pol_w);
                        else pair_load_3d(sa + i * bbytes, &map_w, k, c0, q.e, bar, pol_w);
                        pair_load_2d(sa + i * bbytes + PA_BYTES, map_rows, k, r0, bar, pol_r);
                    }
                }
                pending |= 1u << stage;
                pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
                if (++stage == stages) { stage = 0; phase ^= 1; }
                if (kb == 0 && j + jstep < jobs) next = job_at(j + jstep, plan, E, NT);   // while these loads fly
            }
        }
        __syncwarp();
        if (rank == 0) pair_drain(bars, pending, pend_par);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader; the warp converged, one lane issues)
        // What this warp executes for a block is dependent instructions of one thread, and has to take less time than the
        // block's products (448 cycles for 224 rows): four blocks at a time with their offsets as constants, and a job's size
        // from the scale warps instead of the work list.
        if (rank == 0) {
            const bool elected = elect_one();
            int stage = 0, job = 0, group = 0;
            uint32_t phase = 0, gphase = 0;
            bool ok = true;
            const uint32_t ring_addr = smem_addr(ring);
            const uint64_t sd0 = scale_desc(smem_addr(scales));
            const uint32_t sf = tmem + (uint32_t)SCALE_COL0;
            for (int j = j0; ok && j < jobs; j += jstep, ++job) {
                uint32_t idesc = 0;
                int pieces = 3;                                  // of scales: the weights', and one or two of the rows'
                const int acc = job & 1;
                const uint32_t d = tmem + (uint32_t)(acc * ACC_COLS);
                if (!pair_wait<true>(&bars->tempty[acc], (uint32_t)((job >> 1) & 1) ^ 1, &bars->abort, status)) break;
                for (int kb0 = 0; ok && kb0 < KB; kb0 += GROUP_KB) {
                    if (!pair_wait<true>(&sbars->full[group], gphase, &bars->abort, status)) { ok = false; break; }
                    if (kb0 == 0) {
                        const int n = *(volatile int*)&sbars->rows[group];
                        idesc = scaled_idesc(n, W_MN);
                        pieces = n > 128 ? 3 : 2;
                    }
                    const uint64_t sd = sd0 + (uint64_t)(group * (GROUP_KB * SCALE_BYTES >> 4));
                    tc_fence_after();
                    if (elected) {                               // behind the MMAs of the group before, in the tensor core's order
#pragma unroll
                        for (int k = 0; k < GROUP_KB; ++k) {
                            if (kb0 + k >= KB) break;
#pragma unroll
                            for (int i = 0; i < 3; ++i)
                                if (i < pieces) copy_scales(sf + k * 12 + i * 4, sd + (uint64_t)((k * SCALE_BYTES + i * SCALE_PIECE) >> 4));
                        }
                        pair_commit(&sbars->empty[group]);
                    }
#pragma unroll
                    for (int h = 0; h < GROUP_KB; h += STAGE_KB) {
                        if (kb0 + h >= KB) break;
                        if (!pair_wait(&bars->full[stage], phase, &bars->abort, status)) { ok = false; break; }
                        tc_fence_after();
                        if (elected) {
#pragma unroll
                            for (int k = h; k < h + STAGE_KB; ++k) {
                                if (kb0 + k >= KB) break;
                                const uint32_t sa = ring_addr + (uint32_t)(stage * sbytes + (k - h) * bbytes);
                                const uint64_t ad = W_MN ? smem_desc_mn8(sa) : smem_desc(sa), bd = smem_desc(sa + PA_BYTES);
#pragma unroll
                                for (int kk = 0; kk < KB8 / UK8; ++kk)   // 32 deep: 32 bytes along a row, 4096 bytes MN-major
                                    scaled_mma(d, ad + (uint64_t)(kk * (W_MN ? 256 : 2)), bd + (uint64_t)(kk * 2), idesc, sf + k * 12,
                                               sf + k * 12 + 4, kk > 0 || k > 0 ? 1u : (uint32_t)kb0);
                            }
                            pair_commit(&bars->empty[stage]);
                        }
                        if (++stage == stages) { stage = 0; phase ^= 1; }
                    }
                    if (++group == GROUPS) { group = 0; gphase ^= 1; }
                }
                if (ok && elected) pair_commit(&bars->tfull[acc]);
            }
            __syncwarp();
            if (elected) pair_commit(&bars->mma_done);
        }
    } else if (warp >= SCALE_WARP) {
        // ------------------------------------------------ scales (both CTAs): lane l has rows l, l + 32, .. of the chunk
        // Each of the warps takes every SCALE_WARPS-th group of the pair's jobs, into a buffer of its own: a turn takes one warp
        // longer than the products of the group's four blocks. The order of a turn matters. The proxy fence waits for everything
        // in flight, so the next group is fetched behind it (in front of it the fence took 1800 to 2900 cycles of the 4000 that
        // two groups last); and finding the next job, some 1500 cycles with 112 experts, comes while those loads fly.
        const int group = warp - SCALE_WARP, NG = (KB + GROUP_KB - 1) / GROUP_KB;
        uint32_t phase = 0;
        const bool words = KB % 4 == 0 && (uintptr_t)row_scales % 4 == 0;
        // A group's bytes, as loaded (a word of a row, or its bytes apart): they are not touched before the next turn, which would
        // wait for them here. 127 (a factor of 1) where there is nothing.
        uint32_t raw_w[GROUP_KB], raw[7][GROUP_KB];
        auto fetch = [&](const Job& q, int kb) {
            const int cb = q.nt * 2 + rank;                      // this CTA's block of output columns
            const uint8_t* wp = w_scales + q.e * ws.per_expert + (int64_t)cb * ws.col_step + (int64_t)kb * ws.k_step;
            const uint8_t* rp = row_scales + (int64_t)(q.row0 + lane) * KB + kb;
            const int left = cb < ws.col_blocks ? KB - kb : 0;
#pragma unroll
            for (int k = 0; k < GROUP_KB; ++k) {
                raw_w[k] = 127u;
                if (k < left) raw_w[k] = __ldg(wp);
                wp += ws.k_step;
            }
            if (words) {
#pragma unroll
                for (int i = 0; i < 7; ++i) {
                    raw[i][0] = 0x7F7F7F7Fu;
                    if (lane + 32 * i < q.rows) raw[i][0] = __ldg((const uint32_t*)rp);
                    rp += 32 * KB;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i) {
#pragma unroll
                    for (int k = 0; k < GROUP_KB; ++k) {
                        raw[i][k] = 127u;
                        if (lane + 32 * i < q.rows && kb + k < KB) raw[i][k] = __ldg(rp + k);
                    }
                    rp += 32 * KB;
                }
            }
        };
        // Groups in order: one whose bytes are here, or on their way (job number, group of the job), and the one after it.
        struct At {
            int j, g;
            Job q;
        };
        auto after = [&](const At& a) {
            At b = a;
            b.g += SCALE_WARPS;
            while (b.g >= NG) {
                b.g -= NG;
                b.j += jstep;
            }
            if (b.j != a.j && b.j < jobs) b.q = job_at(b.j, plan, E, NT);
            return b;
        };
        At next = {j0 - jstep, NG - SCALE_WARPS + group, Job{}};  // as if behind the job before the first
        next = after(next);
        At here = next;
        if (here.j < jobs) {
            fetch(here.q, here.g * GROUP_KB);
            next = after(here);
        }
        uint8_t* at = scales + group * GROUP_KB * SCALE_BYTES + lane * 16;
        const uint32_t full = cluster_addr(&sbars->full[group], 0);
        while (here.j < jobs) {
            const int blocks = min(GROUP_KB, KB - here.g * GROUP_KB), rows = here.q.n;
            uint32_t b[7];
            const uint32_t wb = bytes4(raw_w[0], raw_w[1], raw_w[2], raw_w[3]);
#pragma unroll
            for (int i = 0; i < 7; ++i) b[i] = words ? raw[i][0] : bytes4(raw[i][0], raw[i][1], raw[i][2], raw[i][3]);
            uint32_t v[GROUP_KB][8];                             // before the wait: what follows it delays the products
#pragma unroll
            for (int k = 0; k < GROUP_KB; ++k) {
#pragma unroll
                for (int i = 0; i < 7; ++i) v[k][i] = __byte_perm(b[i], 0, k * 0x1111);
                v[k][7] = __byte_perm(wb, 0, k * 0x1111);
            }
            if (!pair_wait(&sbars->empty[group], phase ^ 1, &bars->abort, status)) break;
            if (lane == 0) sbars->rows[group] = rows;
#pragma unroll
            for (int k = 0; k < GROUP_KB; ++k) {
                if (k >= blocks) break;
                st_shared_v4(at + k * SCALE_BYTES, v[k][7], v[k][7], v[k][7], v[k][7]);
                st_shared_v4(at + k * SCALE_BYTES + SCALE_PIECE, v[k][0], v[k][1], v[k][2], v[k][3]);
                if (rows > 128) st_shared_v4(at + k * SCALE_BYTES + 2 * SCALE_PIECE, v[k][4], v[k][5], v[k][6], 0x7F7F7F7Fu);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(full);
            phase ^= 1;
            here = next;
            if (here.j < jobs) {
                fetch(here.q, here.g * GROUP_KB);
                next = after(here);
            }
        }
    } else {
        linear_epilogue<ACT>(bars, plan, tmem, ACC_COLS, patches, bias, residual, out, out_fp32, pre, status, E, NCOL, NT, j0,
                             jstep, jobs, rank);
    }
    pair_teardown(tmem, bars);
}

// ---------------------------------------------------------------- few rows per expert

// A decoding step: the read of the weights is the whole cost. A job is 16 weight rows and all rows of one expert, FEW_ROWS at
// most (the launch takes no more rows in all; linear_few_kernel, which does, cuts an expert's into several jobs), the warps of a block share the contraction in steps of 256 (two scale blocks), and
// the products run on mma.m16n8k16 with the codes as fp16, which holds every E4M3 number. A lane's 16-byte
// loads of weights and of the row at the same place are the fragments of four steps, the contraction's order being
// free within a block. A block's sum is multiplied by its scales as it is added to the fp32 total.
constexpr int FEW_WARPS = 8;
constexpr int FEW_ROWS = 16;                 // 1 or 2 tiles of 8

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes as fp16.
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}

// x·2^(ea + ew - 254): in two factors, since their product may leave fp32 where the result does not.
__device__ __forceinline__ float2 scale_factors(uint32_t ea, uint32_t ew) {
    const int e = (int)(ea + ew) - 254;
    const int first = max(-126, min(127, e)), second = max(-126, min(127, e - first));
    float2 f = make_float2(__uint_as_float((uint32_t)(first + 127) << 23), __uint_as_float((uint32_t)(second + 127) << 23));
    if (ea == 255 || ew == 255) f.x = __uint_as_float(0x7FFFFFFFu);
    return f;
}

struct FewShared {
    float part[FEW_WARPS][FEW_ROWS][17];     // [warp][row][weight row], padded
};

template <int NTT>
__device__ __forceinline__ void few_job(FewShared& sh, const uint8_t* a, const uint8_t* as, const uint8_t* we,
                                        const uint8_t* ws, int64_t row0, int rows, int64_t n0, int64_t N, int64_t K, int KB) {
    constexpr int U = 4;                     // loads of 64 elements in flight: two scale blocks of each weight row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = (lane & 3) * 16;
    const uint8_t* w0 = n0 + g < N ? we + (n0 + g) * K : nullptr;
    const uint8_t* w1 = n0 + g + 8 < N ? we + (n0 + g + 8) * K : nullptr;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float total[NTT][4] = {};
    for (int64_t k0 = warp * 256; k0 < K; k0 += FEW_WARPS * 256) {
        uint4 wa[U], wb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + 64 * u + q;
            Vec<4> x{{0, 0, 0, 0}}, y{{0, 0, 0, 0}};
            if (k < K && w0) x = ld_stream<4, true>((const Vec<4>*)(w0 + k));
            if (k < K && w1) y = ld_stream<4, true>((const Vec<4>*)(w1 + k));
            wa[u] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
            wb[u] = make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {        // scale blocks
            const int kb = (int)(k0 >> 7) + h;
            if (kb >= KB) break;
            const uint32_t ew = __ldg(ws + kb);
            float acc[NTT][4] = {};
#pragma unroll
            for (int u = 2 * h; u < 2 * h + 2; ++u) {
                const int64_t k = k0 + 64 * u + q;
                const uint32_t* x = (const uint32_t*)&wa[u];
                const uint32_t* y = (const uint32_t*)&wb[u];
                uint4 t[NTT];
#pragma unroll
                for (int i = 0; i < NTT; ++i)
                    t[i] = (k < K && 8 * i + g < rows) ? __ldg((const uint4*)(a + (row0 + 8 * i + g) * K + k)) : zero;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t a0 = half2_of(x[s]), a2 = half2_of(x[s] >> 16);
                    const uint32_t a1 = half2_of(y[s]), a3 = half2_of(y[s] >> 16);
#pragma unroll
                    for (int i = 0; i < NTT; ++i) {
                        const uint32_t v = ((const uint32_t*)&t[i])[s];
                        mma_f16(acc[i], a0, a1, a2, a3, half2_of(v), half2_of(v >> 16));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NTT; ++i) {  // acc: (weight row g, rows 2(lane % 4), +1), (weight row g + 8, ..)
                const int r = 8 * i + 2 * (lane & 3);
                const float2 f0 = scale_factors(r < rows ? __ldg(as + (row0 + r) * KB + kb) : 127u, ew);
                const float2 f1 = scale_factors(r + 1 < rows ? __ldg(as + (row0 + r + 1) * KB + kb) : 127u, ew);
                total[i][0] += acc[i][0] * f0.x * f0.y;
                total[i][1] += acc[i][1] * f1.x * f1.y;
                total[i][2] += acc[i][2] * f0.x * f0.y;
                total[i][3] += acc[i][3] * f1.x * f1.y;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NTT; ++i) {
        const int r = 8 * i + 2 * (lane & 3);
        sh.part[warp][r][g] = total[i][0];
        sh.part[warp][r + 1][g] = total[i][1];
        sh.part[warp][r][g + 8] = total[i][2];
        sh.part[warp][r + 1][g + 8] = total[i][3];
    }
}

template <int ACT>
__global__ void __launch_bounds__(FEW_WARPS * 32, 3)
    linear_fp8_few_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ as, const uint8_t* __restrict__ w,
                          const uint8_t* __restrict__ ws, const int64_t* __restrict__ offsets, const float* __restrict__ bias,
                          const uint16_t* __restrict__ residual, void* __restrict__ out, int out_fp32,
                          uint16_t* __restrict__ pre, int E, int64_t R, int64_t N, int64_t K) {
    __shared__ FewShared sh;
    __shared__ int owners[MAX_EXPERTS + 1];  // experts with rows before e
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    dependents_wait();
    if (threadIdx.x == 0) owners[0] = 0;
    const bool orderly = each_expert(offsets, E, R, [&](int e, int64_t b, int64_t en) { owners[e + 1] = en > b ? 1 : 0; });
    if (!orderly) drop_overlapping(offsets, E, R, owners + 1, nullptr);
    if (warp == 0) prefix_in_place(owners, E, lane);
    __syncthreads();
    const int T = owners[E];
    const int groups = (int)((N + 15) / 16), KB = (int)((K + KB8 - 1) / KB8), NB = (int)((N + QBLOCK - 1) / QBLOCK);
    const int64_t jobs = (int64_t)T * groups;
    for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int t = (int)(j / groups);
        const int64_t n0 = (int64_t)(j - (int64_t)t * groups) * 16;
        int lo = 0, hi = E - 1;              // last e with owners[e] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (owners[mid] <= t) lo = mid; else hi = mid - 1;
        }
        int64_t row0, end;
        expert_range(offsets, lo, R, row0, end);
        const int rows = (int)(end - row0);
        const uint8_t* we = w + (int64_t)lo * N * K;
        const uint8_t* se = ws + ((int64_t)lo * NB + n0 / QBLOCK) * KB;
        if (rows <= 8) few_job<1>(sh, a, as, we, se, row0, rows, n0, N, K, KB);
        else few_job<2>(sh, a, as, we, se, row0, rows, n0, N, K, KB);
        __syncthreads();
        for (int i = threadIdx.x; i < rows * 16; i += blockDim.x) {
            const int r = i >> 4, c = i & 15;
            const int64_t n = n0 + c;
            if (n >= N) continue;
            float z = 0.0f;
#pragma unroll
            for (int k = 0; k < FEW_WARPS; ++k) z += sh.part[k][r][c];
            if (bias) z += bias[(int64_t)lo * N + n];
            const int64_t at = (row0 + r) * N + n;
            if (pre) pre[at] = f32_to_bf16(z);
            float y = act_value<ACT>(z);
            if (residual) y += bf16_to_f32(residual[at]);
            if (out_fp32) ((float*)out)[at] = y;
            else ((uint16_t*)out)[at] = f32_to_bf16(y);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- host side

// What linear_fp8_few_kernel takes of the forward: few rows, and weights that a few SMs' tiles would not stream at HBM's rate.
// (few / tensor-core kernel, us. One weight of 3584 x 3584: 1 row 6.4 / 11.4, 16 rows 8.6 / 12.1, 32 rows 14.4 / 12.1; of
// 14336 x 3584: 1 row 13.0 / 16.0. 112 experts of 3584 x 2048: 8 rows 18.2 / 13.9, 128 rows 126 / 83, 448 rows 202 / 128; 8
// experts of 1024 x 1024: 8 rows 5.2 / 8.3.)
constexpr int64_t FEW_MAX_ROWS = 16;
static_assert(FEW_MAX_ROWS <= FEW_ROWS, "an expert's rows are one job");
constexpr int64_t FEW_MAX_WEIGHTS = 52 << 20;

struct Args {
    const uint8_t *a, *as, *w, *ws;
    const int64_t* offsets;
    int64_t E;
    const float* bias;
    const void* residual;
    void* out;
    bool out_fp32;
    void* pre;
    int* status;
    int64_t R, N, K;
    cudaStream_t stream;
};

// NCOL output columns (N forward, K dgrad), KC the contraction.
template <bool W_MN, int ACT>
int launch_tc(const Args& p) {
    const int64_t NCOL = W_MN ? p.K : p.N, KC = W_MN ? p.N : p.K;
    CUtensorMap map_w;
    RowMaps map_r;
    const uint64_t rdims[2] = {(uint64_t)KC, (uint64_t)p.R}, rstride[1] = {(uint64_t)KC};
    for (uint32_t i = 0; i < ROW_MAPS; ++i) {
        const uint32_t box[2] = {KB8, 16 * (i + 1)};
        if (!make_map_bytes(&map_r.m[i], p.a, 2, rdims, rstride, box, CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
            return cuda_fail(cudaErrorInvalidValue);
    }
    // [E, N, K] as stored
    const uint64_t dims[3] = {(uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.E}, strides[2] = {(uint64_t)p.K, (uint64_t)(p.N * p.K)};
    const uint32_t box[3] = {128, 128, 1};
    const CUtensorMapL2promotion promo = p.K % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    if (!make_map_bytes(&map_w, p.w, 3, dims, strides, box, promo)) return cuda_fail(cudaErrorInvalidValue);
    int sms = 0;
    const int st = sm_count(&sms);
    if (st != SITU_GLU_OK) return st;
    const int NT = (int)((NCOL + TILE - 1) / TILE);
    const int64_t KB = (KC + KB8 - 1) / KB8;
    const int most = pick_chunk(p.R, p.E, NT, KB, sms / 2, MAX_CHUNK);
    const int64_t jobs = ((p.R + most - 1) / most + p.E - 1) * NT;   // at most: every expert's last chunk partial
    if (jobs > INT32_MAX - 2 * sms) return SITU_GLU_INVALID_ARG;     // the kernel counts them in 32 bits
    const int nb = (int)((p.N + QBLOCK - 1) / QBLOCK), kb = (int)((p.K + QBLOCK - 1) / QBLOCK);
    const ScaleStrides ss = {(int64_t)nb * kb, W_MN ? 1 : kb, W_MN ? kb : 1, W_MN ? kb : nb};
    const cudaError_t e = launch_pairs<true>(linear_fp8_tc_kernel<W_MN, ACT>, jobs, NUM_THREADS, SMEM_BYTES, p.stream, map_w, map_r, p.as,
                                       p.ws, ss, p.offsets, p.bias, (const uint16_t*)p.residual, p.out, p.out_fp32 ? 1 : 0,
                                       (uint16_t*)p.pre, p.status, (int)p.E, p.R, NCOL, (int)KB, most);
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

template <int ACT>
int launch_few(const Args& p) {
    auto kernel = linear_fp8_few_kernel<ACT>;
    // one warp of work per row as grid_for counts it: every 16 weight rows of every expert that may have rows
    int grid = 0;
    const int64_t experts = p.R < p.E ? p.R : p.E;
    const int st = grid_for((const void*)kernel, FEW_WARPS * 32, experts * ((p.N + 15) / 16) * FEW_WARPS, &grid);
    if (st != SITU_GLU_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(FEW_WARPS * 32);
    cfg.stream = p.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p.a, p.as, p.w, p.ws, p.offsets, p.bias, (const uint16_t*)p.residual, p.out,
                                             p.out_fp32 ? 1 : 0, (uint16_t*)p.pre, (int)p.E, p.R, p.N, p.K);
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

template <int ACT>
int launch_fwd(const Args& p) {
    const int64_t experts = p.R < p.E ? p.R : p.E;       // with rows, at most
    return p.R <= FEW_MAX_ROWS && p.N * p.K <= FEW_MAX_WEIGHTS / experts ? launch_few<ACT>(p) : launch_tc<false, ACT>(p);
}

int check_fp8(int64_t E, const void* offsets, int64_t R, int64_t N, int64_t K) {
    if (N % 16 != 0 || K % 16 != 0) return SITU_GLU_INVALID_ARG;     // TMA: rows of codes are multiples of 16 bytes
    return check_linear(E, offsets, R, N, K);
}

int64_t nblocks(int64_t n) { return (n + QBLOCK - 1) / QBLOCK; }

}  // namespace

extern "C" {

int situ_linear_fp8_fwd(const uint8_t* a, const uint8_t* a_scales, const uint8_t* w, const uint8_t* w_scales,
                        const int64_t* expert_offsets, int64_t E, const float* bias, const void* residual, int act, void* out,
                        int out_type, void* pre, int* status, int64_t R, int64_t N, int64_t K, cudaStream_t stream) {
    const int st = check_fp8(E, expert_offsets, R, N, K);
    if (st != SITU_GLU_OK) return st;
    if (act < SITU_ACT_NONE || act > SITU_ACT_GELU || (out_type != SITU_BF16 && out_type != SITU_FP32))
        return SITU_GLU_INVALID_ARG;
    if (R == 0) return SITU_GLU_OK;
    if (!a || !a_scales || !w || !w_scales || !out) return SITU_GLU_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(residual, 16) || !aligned(pre, 16) ||
        !aligned(bias, 4) || !aligned(expert_offsets, 8) || !aligned(status, 4))
        return SITU_GLU_INVALID_ARG;
    const int64_t osz = out_type == SITU_FP32 ? 4 : 2;
    const Range in[7] = {range_of(a, R * K), range_of(a_scales, R * nblocks(K)), range_of(w, E * N * K),
                         range_of(w_scales, E * nblocks(N) * nblocks(K)), range_of(bias, bias ? E * N * 4 : 0),
                         range_of(residual, residual ? R * N * 2 : 0),
                         range_of(expert_offsets, expert_offsets ? (E + 1) * 8 : 0)};
    const Range o[3] = {range_of(out, R * N * osz), range_of(pre, pre ? R * N * 2 : 0), range_of(status, status ? 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (overlap(o[i], r)) return SITU_GLU_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(o[i], o[j])) return SITU_GLU_OVERLAP;
    }
    const Args p = {a, a_scales, w, w_scales, expert_offsets, E, bias, residual, out, out_type == SITU_FP32, pre, status, R, N, K, stream};
    switch (act) {
        case SITU_ACT_RELU: return launch_fwd<SITU_ACT_RELU>(p);
        case SITU_ACT_SILU: return launch_fwd<SITU_ACT_SILU>(p);
        case SITU_ACT_GELU: return launch_fwd<SITU_ACT_GELU>(p);
        default: return launch_fwd<SITU_ACT_NONE>(p);
    }
}

int situ_linear_fp8_dgrad(const uint8_t* dz, const uint8_t* dz_scales, const uint8_t* w, const uint8_t* w_scales,
                          const int64_t* expert_offsets, int64_t E, void* da, int* status, int64_t R, int64_t N, int64_t K,
                          cudaStream_t stream) {
    const int st = check_fp8(E, expert_offsets, R, N, K);
    if (st != SITU_GLU_OK) return st;
    if (R == 0) return SITU_GLU_OK;
    if (!dz || !dz_scales || !w || !w_scales || !da) return SITU_GLU_INVALID_ARG;
    if (!aligned(dz, 16) || !aligned(w, 16) || !aligned(da, 16) || !aligned(expert_offsets, 8) || !aligned(status, 4))
        return SITU_GLU_INVALID_ARG;
    const Range rda = range_of(da, R * K * 2), rs = range_of(status, status ? 4 : 0);
    for (const Range& r : {range_of(dz, R * N), range_of(dz_scales, R * nblocks(N)), range_of(w, E * N * K),
                           range_of(w_scales, E * nblocks(N) * nblocks(K)),
                           range_of(expert_offsets, expert_offsets ? (E + 1) * 8 : 0)})
        if (overlap(rda, r) || overlap(rs, r)) return SITU_GLU_OVERLAP;
    if (overlap(rda, rs)) return SITU_GLU_OVERLAP;
    return launch_tc<true, SITU_ACT_NONE>({dz, dz_scales, w, w_scales, expert_offsets, E, nullptr, nullptr, da, false, nullptr,
                                           status, R, N, K, stream});
}

}  // extern "C"
