// situ_linear.cu — matrix product of every row with its expert's (or the one dense) weight, with
// bias, activation and residual in the epilogue, and the input gradient (include/situ_moe.h).
//
//   forward   out[r] = act(a[r]·W_eᵀ + b_e) + residual[r]
//   dgrad     da[r]  = dz[r]·W_e
//
// Two kernels:
//   * linear_tc_kernel: tcgen05 on pairs of SMs (situ_pair.cuh). The WEIGHTS are the MMA's 256-row operand and
//     the rows its N operand: an accumulator is (256 output columns) x (up to 256 rows of one expert), and as
//     N may be any multiple of 32, an expert's ragged rows cost what they are, not a multiple of 128. The
//     transposed accumulator suits the epilogue too: a lane holds one output column, so the bias is one
//     value and a warp's stores (and residual loads) of a row are 64 consecutive bytes, whatever the
//     number of rows. Weights are a 3-D tensor [E, N, K], so the boxes of a ragged edge read zeros, never
//     the next expert; rows past a chunk's end are computed and not stored.
//   * linear_few_kernel: for few rows per expert (a decoding step), where the weights' one trip from
//     HBM is the whole cost: see there.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/situ_moe.h"
#include "situ_device.cuh"
#include "situ_host.h"
#include "situ_linear.cuh"
#include "situ_pair.cuh"

namespace {

using namespace situ;
using namespace situ_host;
using namespace situ_pair;
using namespace situ_linear;

constexpr int EPW = 2;                       // epilogue warps per 32-lane TMEM quadrant
constexpr int CW = 32;                       // rows (accumulator columns) per epilogue step
constexpr int PATCH = CW * 64;               // 32 rows x 32 output columns of bf16 in shared memory, per warp
constexpr int NUM_EPI_WARPS = 4 * EPW;
constexpr int NUM_THREADS = 64 + NUM_EPI_WARPS * 32;  // warp 0 TMA, warp 1 MMA, then the epilogue
constexpr int TILE = 256;                    // output columns per job: 128 per CTA of the pair
constexpr int MAX_CHUNK = 256;               // rows per job: the MMA's largest N
constexpr int GROUP = 8;                     // chunks of an expert worked on at a time

// A ring stage: 128 weight rows and half of the chunk's rows, 128 bytes each.
__host__ __device__ constexpr int stage_bytes(int most) { return PA_BYTES + most / 2 * 128; }
__host__ __device__ constexpr int ring_stages(int most) {
    const int s = PRING_BYTES / stage_bytes(most);
    return s < PSTAGES ? s : PSTAGES;
}
static_assert(ring_stages(MAX_CHUNK) == 6 && ring_stages(192) == 7, "ring");

struct Job {
    int e, nt;
    int row0;                                // first row of the chunk
    int rows;                                // rows of the chunk
    int n;                                   // rows rounded up to the MMA's multiple of 32
};

// The work list, in shared memory: an expert's rows are cut into chunks of at most `most` rows (a multiple of
// 32), as even as multiples of 32 allow; a job is one chunk times one tile of output columns.
struct Plan {
    int start[MAX_EXPERTS + 1];              // chunks of the experts before e
    int begin[MAX_EXPERTS];                  // first row of e
    int rows[MAX_EXPERTS];
};

// Job j: the experts in order; within one, GROUP chunks at a time, and within those the output tiles in
// order, so that the pairs at work at one time share a few weight tiles and a few chunks. 32-bit throughout
// (the host bounds the number of jobs): with 64-bit divisions and offsets from global memory, finding the next
// job took longer than the ring holds work, 0.8 us of every job.
__device__ __forceinline__ Job job_at(int j, const Plan& plan, int E, int NT) {
    int lo = 0, hi = E - 1;                  // last e whose first job is <= j
    const int ch = j / NT;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (plan.start[mid] <= ch) lo = mid; else hi = mid - 1;
    }
    Job q;
    q.e = lo;
    const int first = plan.start[lo], nch = plan.start[lo + 1] - first;
    const int local = j - first * NT;
    const int g = local / (GROUP * NT), rem = local - g * (GROUP * NT);
    const int width = min(GROUP, nch - g * GROUP);
    q.nt = rem / width;
    const int c = g * GROUP + rem - q.nt * width;
    const int size = ((plan.rows[lo] - 1) / nch + 32) & ~31;   // no sum that could pass 2^31
    q.row0 = plan.begin[lo] + c * size;
    q.rows = min(size, plan.rows[lo] - c * size);
    q.n = (q.rows + 31) & ~31;
    return q;
}

constexpr int SMEM_BYTES = 1024 + PRING_BYTES + NUM_EPI_WARPS * PATCH + (int)sizeof(PairBars) + (int)sizeof(Plan);
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

// ---- the epilogue's layouts. The accumulator is (output columns) x (rows), memory is rows x columns. tcgen05.ld
// 16x256b gives a lane two rows of one output column, the fragment of 8 x 8 matrices that stmatrix transposes on
// its way to shared memory: a warp's patch of 32 rows x 32 columns (64 bytes a row) takes 4 stmatrix and
// leaves in 4 coalesced 16-byte stores a lane. (2-byte stores straight from a column's lane, 64 bytes a
// store, cost 6 cycles each: 6000 cycles for a 256-row accumulator, more than its products at K = 768.)
// The residual comes the same way back, through ldmatrix.
__device__ __forceinline__ void tc_ld_16x256(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Byte of the 16-byte piece g (of 4) of row i in a patch: swizzled so that neither eight consecutive rows' pieces
// (stmatrix, ldmatrix) nor eight lanes' 16-byte accesses share banks.
__device__ __forceinline__ uint32_t patch_at(int i, int g) { return (uint32_t)(i * 64 + ((g ^ ((i >> 1) & 3)) << 4)); }

__device__ __forceinline__ void st_matrix_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void ld_matrix_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// A patch between shared memory and rows of NCOL elements in global memory: lane l moves the piece l % 4 of rows
// l / 4, l / 4 + 8, .. `at`: the element of the patch's row 0, column 0; ncols: columns inside the matrix
// (a multiple of 8).
__device__ __forceinline__ void patch_out(const uint8_t* patch, uint16_t* out, int64_t at, int64_t NCOL, int left, int ncols,
                                          int lane) {
#pragma unroll
    for (int i = lane >> 2; i < CW; i += 8) {
        const uint4 v = *(const uint4*)(patch + patch_at(i, lane & 3));
        if (i < left && (lane & 3) * 8 < ncols)
            st_stream<4>((Vec<4>*)(out + at + (int64_t)i * NCOL + (lane & 3) * 8), Vec<4>{{v.x, v.y, v.z, v.w}});
    }
}

// W_MN: A is W_eᵀ (dgrad), read MN-major from W_e as stored. ACT: the activation. NCOL output columns
// (N forward, K dgrad), KB 64-deep blocks of the contraction. map_r[i]: the rows' tensor with boxes of
// 128 >> i rows.
struct RowMaps {
    CUtensorMap m[4];
};

template <bool W_MN, int ACT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_r,
                     const int64_t* __restrict__ offsets, const float* __restrict__ bias,
                     const uint16_t* __restrict__ residual, void* __restrict__ out, int out_fp32,
                     uint16_t* __restrict__ pre, int* __restrict__ status, int E, int64_t R, int64_t NCOL, int KB,
                     int most) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* patches = ring + PRING_BYTES;
    PairBars* bars = (PairBars*)(patches + NUM_EPI_WARPS * PATCH);
    Plan& plan = *(Plan*)(bars + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int NT = (int)((NCOL + TILE - 1) / TILE);
    const int sbytes = stage_bytes(most), stages = ring_stages(most);

    if (threadIdx.x == 0) plan.start[0] = 0;
    const bool orderly = each_expert(offsets, E, R, [&](int e, int64_t b, int64_t en) {
        plan.begin[e] = (int)b;
        plan.rows[e] = (int)(en - b);
        plan.start[e + 1] = (int)((en - b + most - 1) / most);
    });
    if (!orderly) drop_overlapping(offsets, E, R, plan.start + 1, plan.rows);
    if (warp == 0) prefix_in_place(plan.start, E, lane);
    const uint32_t tmem = pair_setup(bars, NUM_EPI_WARPS);
    const int jobs = plan.start[E] * NT;
    const int j0 = blockIdx.x >> 1, jstep = gridDim.x >> 1;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs; the warp converged, one lane issues)
        const bool elected = elect_one();
        int stage = 0;
        uint32_t phase = 0, pending = 0, pend_par = 0;
        const uint64_t pol_w = make_policy<kHintB>(), pol_r = make_policy<kHintA>();
        bool ok = true;
        Job next = {};
        if (j0 < jobs) next = job_at(j0, plan, E, NT);
        for (int j = j0; ok && j < jobs; j += jstep) {
            const Job q = next;
            const int c0 = q.nt * TILE + rank * 128;
            const uint32_t bytes = (uint32_t)(2 * PA_BYTES + q.n * 128);
            for (int kb = 0; kb < KB; ++kb) {
                if (!pair_wait(&bars->empty[stage], phase ^ 1, &bars->abort, status)) { ok = false; break; }
                if (elected) {
                    if (rank == 0) mbar_expect_tx(&bars->full[stage], bytes);
                    const uint32_t bar = cluster_addr(&bars->full[stage], 0);
                    uint8_t* sa = ring + stage * sbytes;
                    if constexpr (W_MN) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            pair_load_3d(sa + i * PBOX_BYTES, &map_w, c0 + 64 * i, kb * BK, q.e, bar, pol_w);
                    } else {
                        pair_load_3d(sa, &map_w, kb * BK, c0, q.e, bar, pol_w);
                    }
                    const int half = q.n >> 1;                   // rows of this CTA: a multiple of 16
                    int at = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (half & (128 >> i)) {
                            pair_load_2d(sa + PA_BYTES + at * 128, &map_r.m[i], kb * BK, q.row0 + rank * half + at, bar, pol_r);
                            at += 128 >> i;
                        }
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
        if (rank == 0) {
            const bool elected = elect_one();
            int stage = 0, job = 0;
            uint32_t phase = 0;
            bool ok = true;
            int n_next = j0 < jobs ? job_at(j0, plan, E, NT).n : 0;
            const uint32_t ring_addr = smem_addr(ring);
            for (int j = j0; ok && j < jobs; j += jstep, ++job) {
                const uint32_t idesc = pair_idesc(n_next, W_MN, false);
                const int acc = job & 1;
                const uint32_t d = tmem + (uint32_t)(acc * 256);
                if (!pair_wait<true>(&bars->tempty[acc], (uint32_t)((job >> 1) & 1) ^ 1, &bars->abort, status)) break;
                tc_fence_after();
                for (int kb = 0; kb < KB; ++kb) {
                    if (!pair_wait(&bars->full[stage], phase, &bars->abort, status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sa = ring_addr + (uint32_t)(stage * sbytes);
                    const uint64_t ad = W_MN ? smem_desc_mn(sa) : smem_desc(sa), bd = smem_desc(sa + PA_BYTES);
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < BK / UK; ++kk)     // 16 deep: 32 bytes along a row, 2048 bytes MN-major
                            pair_mma(d, ad + (uint64_t)(kk * (W_MN ? 128 : 2)), bd + (uint64_t)(kk * 2), idesc,
                                     kk > 0 ? 1u : (uint32_t)kb);
                        pair_commit(&bars->empty[stage]);
                    }
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                    if (kb == 0 && j + jstep < jobs) n_next = job_at(j + jstep, plan, E, NT).n;   // while these run
                }
                if (ok && elected) pair_commit(&bars->tfull[acc]);
            }
            __syncwarp();
            if (elected) pair_commit(&bars->mma_done);
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        const int quad = warp & 3;
        const int slot = (warp - 2) >> 2;
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        uint8_t* patch = patches + (warp - 2) * PATCH;
        const uint32_t patch_addr = smem_addr(patch);
        int job = 0;
        for (int j = j0; j < jobs; j += jstep, ++job) {
            const Job q = job_at(j, plan, E, NT);
            const int64_t col = (int64_t)q.nt * TILE + rank * 128 + quad * 32;   // the warp's 32 columns
            const int ncols = (int)max((int64_t)0, min((int64_t)32, NCOL - col));
            float b[4];                                          // bias of this lane's columns: lane / 4 + 8 i
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = (lane >> 2) + 8 * i;
                b[i] = bias && c < ncols ? __ldg(bias + (int64_t)q.e * NCOL + col + c) : 0.0f;
            }
            const int acc = job & 1;
            // residual pieces of the next patch, fetched a patch ahead
            Vec<4> res[4];
            auto fetch_residual = [&](int c) {
                if (residual && ncols > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = c + (lane >> 2) + 8 * i;
                        if (r < q.rows && (lane & 3) * 8 < ncols)
                            res[i] = ld_stream<4, true>((const Vec<4>*)(residual + (int64_t)(q.row0 + r) * NCOL + col + (lane & 3) * 8));
                    }
                }
            };
            fetch_residual(slot * CW);
            const bool ok = pair_wait_epilogue(&bars->tfull[acc], (uint32_t)((job >> 1) & 1), bars, status, NUM_EPI_WARPS);
#pragma unroll 1
            for (int c = slot * CW; c < q.rows; c += EPW * CW) {
                if (!ok) break;
                const int left = q.rows - c;                   // uniform over the warp
                const int64_t at = (int64_t)(q.row0 + c) * NCOL + col;
                uint32_t v[2][16];                           // [columns 0-15, 16-31][8 rows: column l / 4 rows 2(l % 4), +1;
                                                             //  column l / 4 + 8 the same]
                tc_ld_16x256(tmem + t_lane + (uint32_t)(acc * 256 + c), v[0]);
                tc_ld_16x256(tmem + t_lane + (16u << 16) + (uint32_t)(acc * 256 + c), v[1]);
                if (residual) {
                    __syncwarp();                            // the patch has been read out
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *(uint4*)(patch + patch_at((lane >> 2) + 8 * i, lane & 3)) = make_uint4(res[i].w[0], res[i].w[1], res[i].w[2], res[i].w[3]);
                    __syncwarp();
                    fetch_residual(c + EPW * CW);
                }
                tc_wait_ld();
                float2 z[4][4];                              // [8-row group][column block: 0, 8, 16, 24] two rows
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        z[g][i] = __fadd2_rn(make_float2(__uint_as_float(v[i >> 1][4 * g + 2 * (i & 1)]),
                                                         __uint_as_float(v[i >> 1][4 * g + 2 * (i & 1) + 1])),
                                             make_float2(b[i], b[i]));
                if (pre) __syncwarp();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint32_t at_g = patch_addr + patch_at(8 * g + (lane & 7), lane >> 3);
                    uint32_t r[4];
                    if (residual) ld_matrix_t(at_g, r);
                    if (pre) {
                        __syncwarp();
                        st_matrix_t(at_g, pack_bf16x2(z[g][0].x, z[g][0].y), pack_bf16x2(z[g][1].x, z[g][1].y),
                                    pack_bf16x2(z[g][2].x, z[g][2].y), pack_bf16x2(z[g][3].x, z[g][3].y));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        z[g][i] = act_pair<ACT>(z[g][i]);
                        if (residual) z[g][i] = __fadd2_rn(z[g][i], make_float2(bf16_lo(r[i]), bf16_hi(r[i])));
                    }
                }
                if (pre) {
                    __syncwarp();
                    patch_out(patch, pre, at, NCOL, left, ncols, lane);
                }
                if (out_fp32) {                              // 8 lanes' columns of a row: 32 bytes
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = 8 * g + 2 * (lane & 3) + (i & 1), cc = (lane >> 2) + 8 * (i >> 1);
                            if (r < left && cc < ncols)
                                ((float*)out)[at + (int64_t)r * NCOL + cc] = i & 1 ? z[g][i >> 1].y : z[g][i >> 1].x;
                        }
                } else {
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        st_matrix_t(patch_addr + patch_at(8 * g + (lane & 7), lane >> 3), pack_bf16x2(z[g][0].x, z[g][0].y),
                                    pack_bf16x2(z[g][1].x, z[g][1].y), pack_bf16x2(z[g][2].x, z[g][2].y),
                                    pack_bf16x2(z[g][3].x, z[g][3].y));
                    __syncwarp();
                    patch_out(patch, (uint16_t*)out, at, NCOL, left, ncols, lane);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(&bars->tempty[acc], 0));   // read: may be overwritten
        }
    }
    pair_teardown(tmem, bars);
}

// ---------------------------------------------------------------- few rows per expert

// A decoding step gives an expert a row or a few: the product is a read of the weights (22 MB an
// expert at 3584 x 3072), so the kernel is built around that read. A job is 16 weight rows (output
// columns) and up to FEW_ROWS rows of one expert; the FEW_WARPS warps of a block share the
// contraction (warp w takes every FEW_WARPS-th 128-wide block), each with its block's 16-byte loads in
// flight, and meet in shared memory at the end. The products run on mma.m16n8k16
// with the weight rows as the 16 and the tokens as the 8 (a 128-row tcgen05 tile would be nearly
// empty): the contraction's order is free, so a lane's 16-byte load of weights and the one of the
// token's row at the same place are used as they come, as the fragments of two steps.
constexpr int FEW_WARPS = 8;
constexpr int FEW_ROWS = 32;                 // rows of one job: 1, 2 or 4 tiles of 8

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return __ldg((const uint4*)p); }

__device__ __forceinline__ uint4 ld16_stream(const uint16_t* p) {
    const Vec<4> v = ld_stream<4, true>((const Vec<4>*)p);
    return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

// Accumulate NTT tiles of 8 rows x 16 weight rows over this warp's share of the contraction. wr: this
// lane's weight rows (lane / 4 and lane / 4 + 8; NULL past N), ar: this lane's row of each tile (NULL
// past the expert's rows), q = (lane % 4)·8 its place in a 32-wide step.
template <int NTT>
__device__ __forceinline__ void few_accumulate(float (&acc)[NTT][4], const uint16_t* w0, const uint16_t* w1,
                                               const uint16_t* const (&ar)[NTT], int64_t K, int k_first, int q) {
    constexpr int U = 4;                     // 32-wide steps in flight: 64 bytes of each weight row
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t k0 = (int64_t)k_first; k0 < K; k0 += FEW_WARPS * 32 * U) {
        uint4 wa[U], wb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + 32 * u + q;
            wa[u] = (k < K && w0) ? ld16_stream(w0 + k) : zero;
            wb[u] = (k < K && w1) ? ld16_stream(w1 + k) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + 32 * u + q;
#pragma unroll
            for (int i = 0; i < NTT; ++i) {
                const uint4 x = (k < K && ar[i]) ? ld16(ar[i] + k) : zero;
                mma_m16n8k16(acc[i], wa[u].x, wb[u].x, wa[u].y, wb[u].y, x.x, x.y);
                mma_m16n8k16(acc[i], wa[u].z, wb[u].z, wa[u].w, wb[u].w, x.z, x.w);
            }
        }
    }
}

struct FewShared {
    float part[FEW_WARPS][FEW_ROWS][17];     // [warp][row][weight row], padded
};

template <int NTT>
__device__ __forceinline__ void few_job(FewShared& sh, const uint16_t* a, const uint16_t* we, int64_t row0, int rows,
                                        int64_t n0, int64_t N, int64_t K) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const uint16_t* w0 = n0 + g < N ? we + (n0 + g) * K : nullptr;
    const uint16_t* w1 = n0 + g + 8 < N ? we + (n0 + g + 8) * K : nullptr;
    const uint16_t* ar[NTT];
    float acc[NTT][4];
#pragma unroll
    for (int i = 0; i < NTT; ++i) {
        ar[i] = 8 * i + g < rows ? a + (row0 + 8 * i + g) * K : nullptr;
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    }
    few_accumulate<NTT>(acc, w0, w1, ar, K, warp * 128, (lane & 3) * 8);
#pragma unroll
    for (int i = 0; i < NTT; ++i) {          // acc: (weight row g, rows 2(lane % 4), +1), (weight row g + 8, ..)
        const int r = 8 * i + 2 * (lane & 3);
        sh.part[warp][r][g] = acc[i][0];
        sh.part[warp][r + 1][g] = acc[i][1];
        sh.part[warp][r][g + 8] = acc[i][2];
        sh.part[warp][r + 1][g + 8] = acc[i][3];
    }
}

template <int ACT>
__global__ void __launch_bounds__(FEW_WARPS * 32, 3)
    linear_few_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ w, const int64_t* __restrict__ offsets,
                      const float* __restrict__ bias, const uint16_t* __restrict__ residual, void* __restrict__ out,
                      int out_fp32, uint16_t* __restrict__ pre, int E, int64_t R, int64_t N, int64_t K) {
    __shared__ FewShared sh;
    __shared__ int tile_start[MAX_EXPERTS + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // first job of each expert: ceil(rows / FEW_ROWS) each
    if (threadIdx.x == 0) tile_start[0] = 0;
    const bool orderly = each_expert(offsets, E, R, [&](int e, int64_t b, int64_t en) {
        tile_start[e + 1] = (int)((en - b + FEW_ROWS - 1) / FEW_ROWS);
    });
    if (!orderly) drop_overlapping(offsets, E, R, tile_start + 1, nullptr);
    if (warp == 0) prefix_in_place(tile_start, E, lane);
    __syncthreads();
    const int T = tile_start[E];
    const int groups = (int)((N + 15) / 16);
    const int64_t jobs = (int64_t)T * groups;
    for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int t = (int)(j / groups);
        const int64_t n0 = (int64_t)(j - (int64_t)t * groups) * 16;
        int lo = 0, hi = E - 1;              // last e with tile_start[e] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
        }
        int64_t b, en;
        expert_range(offsets, lo, R, b, en);
        const int64_t row0 = b + (int64_t)(t - tile_start[lo]) * FEW_ROWS;
        const int rows = (int)min((int64_t)FEW_ROWS, en - row0);
        const uint16_t* we = w + (int64_t)lo * N * K;
        if (rows <= 8) few_job<1>(sh, a, we, row0, rows, n0, N, K);
        else if (rows <= 16) few_job<2>(sh, a, we, row0, rows, n0, N, K);
        else few_job<4>(sh, a, we, row0, rows, n0, N, K);
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

// Up to how many rows linear_few_kernel takes the forward: on average two an expert, or 64 in all. 112 experts,
// 3584 x 3072 (few / tensor-core kernel): 128 rows 244 / 249 us, 224 rows 327 / 333, 448 rows 369 / 361, 896 rows
// 415 / 378; one weight: 1 row 7.0 / 14.6 us, 32 rows 11.5 / 14.7, 64 rows 14.2 / 14.4, 128 rows 24.7 / 14.6.
constexpr int64_t FEW_MAX_MEAN_ROWS = 2;
constexpr int64_t FEW_MAX_ROWS = 64;

// Most rows per job. A job of n rows takes a 64-deep block in the larger of 2n cycles (tensor cores) and the time
// its (256 + n)·64 bytes per SM need at ~50 bytes a cycle (measured), and jobs run in rounds over the pairs of
// SMs: 256 rows for large shapes, less where that would leave pairs without a job or a round mostly empty. A ring
// stage is sized for them: with weights streamed from HBM the loads in flight count (112 experts of ~292 rows: five
// 32 KB stages 562 us, six 523).
int64_t block_cycles(int64_t n) {
    const int64_t bytes = (256 + n) * 64 / 50;
    return 2 * n > bytes ? 2 * n : bytes;
}

int pick_chunk(int64_t R, int64_t E, int NT, int64_t KB, int pairs) {
    const int64_t rows = (R + E - 1) / E;    // of an expert, on average
    int best = MAX_CHUNK;
    int64_t best_cost = INT64_MAX;
    for (int most = MAX_CHUNK; most >= 32; most -= 32) {
        const int64_t chunks = (rows + most - 1) / most, n = ((rows + chunks - 1) / chunks + 31) / 32 * 32;
        const int64_t last = (rows - (chunks - 1) * n + 31) / 32 * 32;       // the last chunk's, computed last
        const int64_t full = E * (last < n ? chunks - 1 : chunks) * NT, part = last < n ? E * NT : 0;
        const int64_t rounds = (full + pairs - 1) / pairs, left = rounds * pairs - full;
        const int64_t more = part > left ? (part - left + pairs - 1) / pairs : 0;
        const int64_t each = KB * block_cycles(n) + 4 * n + 1500, tail = KB * block_cycles(last) + 4 * last + 1500;
        // many rounds even out over ragged experts; few do not
        const int64_t cost = rounds >= 16 ? (full * each + part * tail) / pairs : rounds * each + more * tail;
        if (cost <= best_cost) {             // of equal chunks the tightest bound: smaller stages, more of them
            best_cost = cost;
            best = most;
        }
    }
    // ragged experts: those with more rows than the average should not be cut for it (each chunk reads the weights again)
    if (E > 1 && E * NT >= pairs) best = 4 * best < MAX_CHUNK ? 4 * best : MAX_CHUNK;
    return best;
}

template <bool W_MN, int ACT>
int launch_tc(const void* a, const void* w, const int64_t* offsets, int64_t E, const float* bias, const void* residual,
              void* out, bool out_fp32, void* pre, int* status, int64_t R, int64_t NCOL, int64_t KC, cudaStream_t stream) {
    CUtensorMap map_w;
    RowMaps map_r;
    for (int i = 0; i < 4; ++i)
        // 128-byte promotion: rows off the 128-byte lines (K = 1000) bring fewer of their neighbours' sectors than with
        // 256 (4099 x 3584 x 1000: 35.0 -> 32.5 us), the others do not care
        if (!make_map(&map_r.m[i], a, (uint64_t)R, (uint64_t)KC, 128u >> i, BK, true, CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
            return cuda_fail(cudaErrorInvalidValue);
    // [E, N, K] as stored; forward: contraction K innermost, dgrad: output columns K innermost
    const uint64_t inner = (uint64_t)(W_MN ? NCOL : KC), rows = (uint64_t)(W_MN ? KC : NCOL);
    const uint64_t dims[3] = {inner, rows, (uint64_t)E}, strides[2] = {inner * 2, inner * rows * 2};
    const uint32_t box[3] = {64, W_MN ? (uint32_t)BK : 128u, 1};
    // weights come from HBM: pieces of 256 bytes where their rows are made of such (the prompt's 534 -> 524 us)
    const CUtensorMapL2promotion promo = inner * 2 % 256 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
    if (!make_map_any(&map_w, w, false, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, promo))
        return cuda_fail(cudaErrorInvalidValue);
    int sms = 0;
    const int st = sm_count(&sms);
    if (st != SITU_GLU_OK) return st;
    const int NT = (int)((NCOL + TILE - 1) / TILE);
    const int64_t KB = (KC + BK - 1) / BK;
    const int most = pick_chunk(R, E, NT, KB, sms / 2);
    const int64_t jobs = ((R + most - 1) / most + E - 1) * NT;   // at most: every expert's last chunk partial
    if (jobs > INT32_MAX - 2 * sms) return SITU_GLU_INVALID_ARG;  // the kernel counts them in 32 bits
    const cudaError_t e = launch_pairs(linear_tc_kernel<W_MN, ACT>, jobs, NUM_THREADS, SMEM_BYTES, stream, map_w, map_r,
                                       offsets, bias, (const uint16_t*)residual, out, out_fp32 ? 1 : 0, (uint16_t*)pre,
                                       status, (int)E, R, NCOL, (int)KB, most);
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

template <int ACT>
int launch_few(const void* a, const void* w, const int64_t* offsets, int64_t E, const float* bias, const void* residual,
               void* out, bool out_fp32, void* pre, int64_t R, int64_t N, int64_t K, cudaStream_t stream) {
    auto kernel = linear_few_kernel<ACT>;
    // one warp of work per row as grid_for counts it: every 16 weight rows of every possible job
    int grid = 0;
    const int64_t tiles = R < E ? R : (R + FEW_ROWS - 1) / FEW_ROWS + E;
    const int st = grid_for((const void*)kernel, FEW_WARPS * 32, tiles * ((N + 15) / 16) * FEW_WARPS, &grid);
    if (st != SITU_GLU_OK) return st;
    kernel<<<grid, FEW_WARPS * 32, 0, stream>>>((const uint16_t*)a, (const uint16_t*)w, offsets, bias,
                                                (const uint16_t*)residual, out, out_fp32 ? 1 : 0, (uint16_t*)pre,
                                                (int)E, R, N, K);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

template <int ACT>
int launch_fwd(const void* a, const void* w, const int64_t* offsets, int64_t E, const float* bias, const void* residual,
               void* out, bool out_fp32, void* pre, int* status, int64_t R, int64_t N, int64_t K, cudaStream_t stream) {
    const bool few = R <= FEW_MAX_ROWS || R <= E * FEW_MAX_MEAN_ROWS;
    return few ? launch_few<ACT>(a, w, offsets, E, bias, residual, out, out_fp32, pre, R, N, K, stream)
               : launch_tc<false, ACT>(a, w, offsets, E, bias, residual, out, out_fp32, pre, status, R, N, K, stream);
}

}  // namespace

extern "C" {

int situ_linear_fwd(const void* a, const void* w, const int64_t* expert_offsets, int64_t E, const float* bias,
                    const void* residual, int act, void* out, int out_type, void* pre, int* status, int64_t R,
                    int64_t N, int64_t K, cudaStream_t stream) {
    const int st = check_linear(E, expert_offsets, R, N, K);
    if (st != SITU_GLU_OK) return st;
    if (act < SITU_ACT_NONE || act > SITU_ACT_GELU || (out_type != SITU_BF16 && out_type != SITU_FP32))
        return SITU_GLU_INVALID_ARG;
    if (R == 0) return SITU_GLU_OK;
    if (!a || !w || !out) return SITU_GLU_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(residual, 16) || !aligned(pre, 16) ||
        !aligned(bias, 4) || !aligned(expert_offsets, 8) || !aligned(status, 4))
        return SITU_GLU_INVALID_ARG;
    const int64_t osz = out_type == SITU_FP32 ? 4 : 2;
    const Range in[5] = {range_of(a, R * K * 2), range_of(w, E * N * K * 2), range_of(bias, bias ? E * N * 4 : 0),
                         range_of(residual, residual ? R * N * 2 : 0),
                         range_of(expert_offsets, expert_offsets ? (E + 1) * 8 : 0)};
    const Range o[3] = {range_of(out, R * N * osz), range_of(pre, pre ? R * N * 2 : 0), range_of(status, status ? 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (overlap(o[i], r)) return SITU_GLU_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(o[i], o[j])) return SITU_GLU_OVERLAP;
    }
    const bool f32 = out_type == SITU_FP32;
    switch (act) {
        case SITU_ACT_RELU: return launch_fwd<SITU_ACT_RELU>(a, w, expert_offsets, E, bias, residual, out, f32, pre, status, R, N, K, stream);
        case SITU_ACT_SILU: return launch_fwd<SITU_ACT_SILU>(a, w, expert_offsets, E, bias, residual, out, f32, pre, status, R, N, K, stream);
        case SITU_ACT_GELU: return launch_fwd<SITU_ACT_GELU>(a, w, expert_offsets, E, bias, residual, out, f32, pre, status, R, N, K, stream);
        default: return launch_fwd<SITU_ACT_NONE>(a, w, expert_offsets, E, bias, residual, out, f32, pre, status, R, N, K, stream);
    }
}

int situ_linear_dgrad(const void* dz, const void* w, const int64_t* expert_offsets, int64_t E, void* da, int* status,
                      int64_t R, int64_t N, int64_t K, cudaStream_t stream) {
    const int st = check_linear(E, expert_offsets, R, N, K);
    if (st != SITU_GLU_OK) return st;
    if (R == 0) return SITU_GLU_OK;
    if (!dz || !w || !da) return SITU_GLU_INVALID_ARG;
    if (!aligned(dz, 16) || !aligned(w, 16) || !aligned(da, 16) || !aligned(expert_offsets, 8) || !aligned(status, 4))
        return SITU_GLU_INVALID_ARG;
    const Range rda = range_of(da, R * K * 2), rs = range_of(status, status ? 4 : 0);
    for (const Range& r : {range_of(dz, R * N * 2), range_of(w, E * N * K * 2),
                           range_of(expert_offsets, expert_offsets ? (E + 1) * 8 : 0)})
        if (overlap(rda, r) || overlap(rs, r)) return SITU_GLU_OVERLAP;
    if (overlap(rda, rs)) return SITU_GLU_OVERLAP;
    return launch_tc<true, SITU_ACT_NONE>(dz, w, expert_offsets, E, nullptr, nullptr, da, false, nullptr, status, R, K,
                                          N, stream);
}

}  // extern "C"
