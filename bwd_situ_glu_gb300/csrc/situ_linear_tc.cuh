// situ_linear_tc.cuh — what the linear operator's tensor-core kernels share, for bf16 operands (situ_linear.cu) and for
// block-scaled 8-bit ones (situ_linear_fp8.cu): the work list of ragged experts, and the epilogue with bias, activation
// and residual. The accumulator is (256 output columns) x (the rows of one chunk), on a pair of SMs (situ_pair.cuh).
#pragma once

#include <stdint.h>

#include "situ_device.cuh"
#include "situ_linear.cuh"
#include "situ_pair.cuh"

namespace situ_linear_tc {

using namespace situ;
using namespace situ_pair;
using namespace situ_linear;

constexpr int EPW = 2;                       // epilogue warps per 32-lane TMEM quadrant
constexpr int CW = 32;                       // rows (accumulator columns) per epilogue step
constexpr int PATCH = CW * 64;               // 32 rows x 32 output columns of bf16 in shared memory, per warp
constexpr int NUM_EPI_WARPS = 4 * EPW;
constexpr int TILE = 256;                    // output columns per job: 128 per CTA of the pair
constexpr int GROUP = 8;                     // chunks of an expert worked on at a time

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

// All threads of a block, then a barrier is due (pair_setup has one): the work list for chunks of at most `most` rows.
__device__ __forceinline__ void build_plan(Plan& plan, const int64_t* offsets, int E, int64_t R, int most) {
    if (threadIdx.x == 0) plan.start[0] = 0;
    const bool orderly = each_expert(offsets, E, R, [&](int e, int64_t b, int64_t en) {
        plan.begin[e] = (int)b;
        plan.rows[e] = (int)(en - b);
        plan.start[e + 1] = (int)((en - b + most - 1) / most);
    });
    if (!orderly) drop_overlapping(offsets, E, R, plan.start + 1, plan.rows);
    if ((threadIdx.x >> 5) == 0) prefix_in_place(plan.start, E, threadIdx.x & 31);
}

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

// The epilogue warps (2 .. NUM_EPI_WARPS + 1) of both CTAs, over the pair's jobs j0, j0 + jstep, ..: accumulator `job & 1` of
// acc_cols TMEM columns, its patch of shared memory per warp at `patches`.
template <int ACT>
__device__ __forceinline__ void linear_epilogue(PairBars* bars, const Plan& plan, uint32_t tmem, int acc_cols, uint8_t* patches,
                                                const float* __restrict__ bias, const uint16_t* __restrict__ residual,
                                                void* __restrict__ out, int out_fp32, uint16_t* __restrict__ pre, int* status,
                                                int E, int64_t NCOL, int NT, int j0, int jstep, int jobs, int rank) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
            tc_ld_16x256(tmem + t_lane + (uint32_t)(acc * acc_cols + c), v[0]);
            tc_ld_16x256(tmem + t_lane + (16u << 16) + (uint32_t)(acc * acc_cols + c), v[1]);
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

// ---------------------------------------------------------------- host side

// Most rows per job, max_chunk at most. A job of n rows takes a 128-byte-deep block (64 of bf16, 128 in 8 bits: twice the
// products in the same time) in the larger of 2n cycles (tensor cores) and the time
// its (256 + n)·64 bytes per SM need at ~50 bytes a cycle (measured of the bf16 product; the 8-bit one has since come to 523 cycles at
// n = 224, 59 bytes a cycle, where this says 614: chunks that large count for a sixth too much there), and jobs run in rounds over the pairs of
// SMs: 256 rows for large shapes, less where that would leave pairs without a job or a round mostly empty. A ring
// stage is sized for them: with weights streamed from HBM the loads in flight count (112 experts of ~292 rows: five
// 32 KB stages 562 us, six 523).
inline int64_t block_cycles(int64_t n) {
    const int64_t bytes = (256 + n) * 64 / 50;
    return 2 * n > bytes ? 2 * n : bytes;
}

inline int pick_chunk(int64_t R, int64_t E, int NT, int64_t KB, int pairs, int max_chunk) {
    const int64_t rows = (R + E - 1) / E;    // of an expert, on average
    int best = max_chunk;
    int64_t best_cost = INT64_MAX;
    for (int most = max_chunk; most >= 32; most -= 32) {
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
    if (E > 1 && E * NT >= pairs) best = 4 * best < max_chunk ? 4 * best : max_chunk;
    return best;
}

}  // namespace situ_linear_tc
