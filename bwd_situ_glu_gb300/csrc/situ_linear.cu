// situ_linear.cu — matrix product of every row with its expert's (or the one dense) weight, with
// bias, activation and residual in the epilogue, and the input gradient (include/situ_moe.h).
//
//   forward   out[r] = act(a[r]·W_eᵀ + b_e) + residual[r]       A = a,  B = W_e  (K-major)
//   dgrad     da[r]  = dz[r]·W_e                                 A = dz, B = W_eᵀ (W_e as stored is N-major)
//
// Two kernels:
//   * linear_tc_kernel: the expert-grouped pipeline of situ_tc.cuh (TMA ring, tcgen05.mma, two TMEM
//     accumulators, bounded waits), whose epilogue adds the bias, applies the activation, adds the
//     residual in fp32 and rounds once. bf16 tiles leave through shared memory as TMA stores (64-byte
//     rows, 64-byte swizzle, so neither the staging writes nor the TMA reads conflict); a quadrant of
//     rows that crosses its expert's end stores from registers. Weights are a 3-D tensor [E, N, K], so
//     the boxes of a ragged edge read zeros, never the next expert.
//   * linear_few_kernel: for few rows per expert (a decoding step), where the weights' one trip from
//     HBM is the whole cost and a 128-row tile would be almost empty: see there.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/situ_moe.h"
#include "situ_device.cuh"
#include "situ_host.h"
#include "situ_linear.cuh"
#include "situ_tc.cuh"

namespace {

using namespace situ;
using namespace situ_host;
using namespace situ_tc;
using namespace situ_linear;

constexpr int EPW = 3;                       // epilogue warps per 32-lane TMEM quadrant
constexpr int CW = 32;                       // accumulator columns per chunk: 64 bytes of bf16
constexpr int NUM_EPI_THREADS = 4 * EPW * 32;
constexpr int NUM_THREADS = 64 + NUM_EPI_THREADS;  // warp 0 TMA, warp 1 MMA, then the epilogue
constexpr int NCH = BN / CW;                 // chunks of a job
constexpr int STAGE_TILE = 32 * CW * 2;      // 32 rows x 64 bytes of output in shared memory
constexpr int SMEM_BYTES = SMEM_FIXED_BYTES + 1024 + 4 * EPW * STAGE_TILE;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

// W_MN: B is W_eᵀ (dgrad; four 64-column boxes per stage). ACT: the activation. NCOL output columns
// (N forward, K dgrad), KB 64-wide blocks of the contraction.
template <bool W_MN, int ACT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_pre,
                     const int64_t* __restrict__ offsets, const float* __restrict__ bias,
                     const uint16_t* __restrict__ residual, void* __restrict__ out, int out_fp32,
                     uint16_t* __restrict__ pre, int* __restrict__ status, int E, int64_t R, int64_t NCOL, int KB,
                     int csplit) {
    extern __shared__ uint8_t smem_raw[];
    const Smem sm = carve_smem(smem_raw);
    Barriers* bars = sm.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NT = (int)((NCOL + BN - 1) / BN);   // the last N-tile may run past NCOL: those columns are
                                                  // products with zeros and never stored
    const Sched sc = make_sched(csplit);
    uint32_t tmem;
    const int T = pipeline_setup(sm, offsets, E, R, NUM_EPI_THREADS, &tmem);

    if (warp == 0) {
        if (lane == 0)
            run_producer(sm, sc, &map_a, offsets, E, R, T, NT, KB, status,
                         [&](uint8_t* sb, int e, int nt, int kb, uint64_t* bar, uint64_t pol) {
                             if constexpr (W_MN) {
#pragma unroll
                                 for (int j = 0; j < BN / 64; ++j)
                                     tma_load_3d_hint(sb + j * BMN_BOX_BYTES, &map_w, nt * BN + 64 * j, kb * BK, e, bar, pol);
                             } else {
                                 tma_load_3d_hint(sb, &map_w, kb * BK, nt * BN, e, bar, pol);
                             }
                         });
    } else if (warp == 1) {
        if (lane == 0) run_mma<W_MN>(sm, sc, tmem, T, NT, KB, status);
    } else {
        const int quad = warp & 3;
        const int slot = (warp - 2) >> 2;
        const int lrow = quad * 32 + lane;
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        uint8_t* stage = (uint8_t*)(((uintptr_t)sm.extra + 1023) & ~(uintptr_t)1023) + (warp - 2) * STAGE_TILE;
        const bool bias_vec = ((uintptr_t)bias & 15) == 0;       // NCOL % 8 == 0 keeps every chunk of it aligned
        bool stores_pending = false;             // lane 0 has TMA stores in flight
        int job = 0;
        bool ok = true;
        // 32 columns of this lane's row as 16 bf16 pairs -> the warp's staged tile -> one TMA store
        auto store_tile = [&](const CUtensorMap* map, const uint32_t (&w)[CW / 2], int col, int row) {
            if (stores_pending) {
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                st_shared_v4(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), w[4 * q], w[4 * q + 1], w[4 * q + 2],
                             w[4 * q + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, col, row, stage);
                bulk_commit();
            }
            stores_pending = true;
        };
        // a job's 32-column chunks are dealt out over the EPW warps of a quadrant: slot, slot + EPW, ..
        // This lane's residual of its next chunk (of this job or the next) is fetched while a chunk is
        // worked off.
        Vec<4> res[4];
        auto fetch_residual = [&](int64_t row0, int64_t row_end, int64_t j0) {
            if (row0 + lrow < row_end) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (j0 + 8 * q < NCOL)
                        res[q] = ld_stream<4, true>((const Vec<4>*)(residual + (row0 + lrow) * NCOL + j0 + 8 * q));
            }
        };
        int e = 0;
        int64_t row0 = 0, row_end = 0;
        if (sc.t0 < T) {
            tile_rows(sm.tile_start, offsets, E, R, sc.t0, e, row0, row_end);
            if (residual) fetch_residual(row0, row_end, (int64_t)sc.n0 * BN + slot * CW);
        }
        for (int t = sc.t0; t < T; t += sc.tstep) {
            int e_next = e;
            int64_t row0_next = row0, row_end_next = row_end;
            if (t + sc.tstep < T) tile_rows(sm.tile_start, offsets, E, R, t + sc.tstep, e_next, row0_next, row_end_next);
            const int64_t row = row0 + lrow;
            const bool full_quad = row0 + quad * 32 + 31 < row_end;
            for (int nt = sc.n0; nt < NT; nt += sc.nstep, ++job) {
                const int acc = job & 1;
                const bool last_job = nt + sc.nstep >= NT;            // of this M-tile
                if (ok && !mbar_wait(&bars->tfull[acc], (uint32_t)((job >> 1) & 1), bars, status)) ok = false;
                ok = __all_sync(FULL_MASK, ok);      // tcgen05.ld below is warp-collective
                const bool valid = ok && row < row_end;
                tc_fence_after();
#pragma unroll 1
                for (int k = slot; k < NCH; k += EPW) {
                    const int64_t j0 = (int64_t)nt * BN + k * CW;
                    const bool chunk = j0 < NCOL;                 // NCOL % 8 == 0: whole groups of 8
                    const bool last = k + EPW >= NCH;
                    float v[CW];
                    if (ok) tc_ld<CW>(tmem + t_lane + (uint32_t)(acc * BN + k * CW), v);
                    if (last) {
                        tc_fence_before();
                        mbar_arrive(&bars->tempty[acc]);          // the accumulator may be overwritten
                    }
                    if (bias && chunk) {
                        // one address for the warp, 16 bytes where the bias allows
                        const float* b = bias + (int64_t)e * NCOL + j0;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (j0 + 4 * q >= NCOL) continue;
                            float4 f;
                            if (bias_vec) f = __ldg((const float4*)(b + 4 * q));
                            else f = make_float4(__ldg(b + 4 * q), __ldg(b + 4 * q + 1), __ldg(b + 4 * q + 2), __ldg(b + 4 * q + 3));
                            v[4 * q] += f.x;
                            v[4 * q + 1] += f.y;
                            v[4 * q + 2] += f.z;
                            v[4 * q + 3] += f.w;
                        }
                    }
                    uint32_t w[CW / 2];
                    if (pre && ok && chunk) {
#pragma unroll
                        for (int i = 0; i < CW / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                        if (full_quad) {
                            store_tile(&map_pre, w, (int)j0, (int)(row0 + quad * 32));
                        } else if (valid) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (j0 + 8 * q < NCOL)
                                    st_stream<4>((Vec<4>*)(pre + row * NCOL + j0 + 8 * q),
                                                 Vec<4>{{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]}});
                        }
                    }
                    if constexpr (ACT != SITU_ACT_NONE) {
#pragma unroll
                        for (int i = 0; i < CW; ++i) v[i] = act_value<ACT>(v[i]);
                    }
                    if (residual) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                v[8 * q + 2 * i] += bf16_lo(res[q].w[i]);      // columns past NCOL and rows past
                                v[8 * q + 2 * i + 1] += bf16_hi(res[q].w[i]);  // the expert are not stored
                            }
                        }
                        if (!last) fetch_residual(row0, row_end, j0 + EPW * CW);
                        else if (!last_job) fetch_residual(row0, row_end, (int64_t)(nt + sc.nstep) * BN + slot * CW);
                        else if (t + sc.tstep < T) fetch_residual(row0_next, row_end_next, (int64_t)sc.n0 * BN + slot * CW);
                    }
                    if (!ok || !chunk) continue;
                    if (out_fp32) {
                        if (valid) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (j0 + 4 * q < NCOL)
                                    st_stream<4>((Vec<4>*)((float*)out + row * NCOL + j0 + 4 * q),
                                                 Vec<4>{{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                                         __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])}});
                        }
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < CW / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                    if (full_quad) {
                        store_tile(&map_out, w, (int)j0, (int)(row0 + quad * 32));
                    } else if (valid) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (j0 + 8 * q < NCOL)
                                st_stream<4>((Vec<4>*)((uint16_t*)out + row * NCOL + j0 + 8 * q),
                                             Vec<4>{{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]}});
                    }
                }
            }
            e = e_next;
            row0 = row0_next;
            row_end = row_end_next;
        }
        if (lane == 0 && stores_pending) bulk_wait_all();   // every staged tile written
    }
    pipeline_teardown(tmem);
}

// ---------------------------------------------------------------- few rows per expert

// A decoding step gives an expert a row or a few: the product is a read of the weights (22 MB an
// expert at 3584 x 3072), so the kernel is built around that read. A job is 16 weight rows (output
// columns) and up to FEW_ROWS rows of one expert; the FEW_WARPS warps of a block share the
// contraction (warp w takes every FEW_WARPS-th 64-wide block), each with its 16-byte loads of
// FEW_U blocks in flight, and meet in shared memory at the end. The products run on mma.m16n8k16
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
__global__ void __launch_bounds__(FEW_WARPS * 32)
    linear_few_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ w, const int64_t* __restrict__ offsets,
                      const float* __restrict__ bias, const uint16_t* __restrict__ residual, void* __restrict__ out,
                      int out_fp32, uint16_t* __restrict__ pre, int E, int64_t R, int64_t N, int64_t K) {
    __shared__ FewShared sh;
    __shared__ int tile_start[MAX_EXPERTS + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // first job of each expert: ceil(rows / FEW_ROWS) each
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int64_t b, en;
        expert_range(offsets, e, R, b, en);
        tile_start[e + 1] = (int)((en - b + FEW_ROWS - 1) / FEW_ROWS);
    }
    if (threadIdx.x == 0) tile_start[0] = 0;
    __syncthreads();
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

// Rows per expert up to which linear_few_kernel takes the forward (see there).
constexpr int64_t FEW_MAX_MEAN_ROWS = 8;
constexpr int64_t FEW_MAX_DENSE_ROWS = 64;

int check_linear(int64_t E, const void* offsets, int64_t R, int64_t N, int64_t K) {
    if (R < 0 || R > INT32_MAX || N < 8 || N % 8 != 0 || K < 8 || K % 8 != 0 || E < 1 || E > MAX_EXPERTS)
        return SITU_GLU_INVALID_ARG;
    if (N > INT32_MAX / 4 || K > INT32_MAX / 4 || E * N > INT32_MAX || E * K > INT32_MAX) return SITU_GLU_INVALID_ARG;
    if (!offsets && E != 1) return SITU_GLU_INVALID_ARG;
    return SITU_GLU_OK;
}

// CTAs sharing an M-tile (its N-tiles dealt out among them): of 4 .. 16, the fewest job rounds for the
// M-tiles expected; more CTAs on a tile at equal rounds keep fewer A tiles live in L2.
int pick_csplit(int64_t R, int64_t E, int NT, int sms) {
    const int64_t tiles = (R + BM - 1) / BM + (E > 1 ? E / 2 : 0);
    int best = NT < 4 ? NT : 4;
    int64_t best_cost = INT64_MAX;
    for (int c = best; c <= NT && c <= 16; ++c) {
        const int groups = sms / c;
        if (groups < 1) break;
        const int64_t cost = ((tiles + groups - 1) / groups) * ((NT + c - 1) / c);
        if (cost <= best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}

template <bool W_MN, int ACT>
int launch_tc(const void* a, const void* w, const int64_t* offsets, int64_t E, const float* bias, const void* residual,
              void* out, bool out_fp32, void* pre, int* status, int64_t R, int64_t NCOL, int64_t KC, cudaStream_t stream) {
    CUtensorMap map_a, map_w, map_out = {}, map_pre = {};
    if (!make_map(&map_a, a, (uint64_t)R, (uint64_t)KC, BM)) return cuda_fail(cudaErrorInvalidValue);
    // [E, N, K] as stored; forward: contraction K innermost, dgrad: output columns K innermost
    const uint64_t inner = (uint64_t)(W_MN ? NCOL : KC), rows = (uint64_t)(W_MN ? KC : NCOL);
    const uint64_t dims[3] = {inner, rows, (uint64_t)E}, strides[2] = {inner * 2, inner * rows * 2};
    const uint32_t box[3] = {64, W_MN ? (uint32_t)BK : (uint32_t)BN, 1};
    if (!make_map_any(&map_w, w, false, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
        return cuda_fail(cudaErrorInvalidValue);
    const uint64_t od[2] = {(uint64_t)NCOL, (uint64_t)R}, os[1] = {(uint64_t)NCOL * 2};
    const uint32_t ob[2] = {CW, 32};
    if (!out_fp32 && !make_map_any(&map_out, out, false, 2, od, os, ob, CU_TENSOR_MAP_SWIZZLE_64B))
        return cuda_fail(cudaErrorInvalidValue);
    if (pre && !make_map_any(&map_pre, pre, false, 2, od, os, ob, CU_TENSOR_MAP_SWIZZLE_64B))
        return cuda_fail(cudaErrorInvalidValue);
    auto kernel = linear_tc_kernel<W_MN, ACT>;
    cudaError_t e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return cuda_fail(e);
    int dev = 0, sms = 0, grid = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const int csplit = pick_csplit(R, E, (int)((NCOL + BN - 1) / BN), sms);
    if ((e = (cudaError_t)persistent_grid(R, E, csplit, &grid)) != cudaSuccess) return cuda_fail(e);
    kernel<<<grid, NUM_THREADS, SMEM_BYTES, stream>>>(map_a, map_w, map_out, map_pre, offsets, bias,
                                                      (const uint16_t*)residual, out, out_fp32 ? 1 : 0, (uint16_t*)pre,
                                                      status, (int)E, R, NCOL, (int)((KC + BK - 1) / BK), csplit);
    e = cudaGetLastError();
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
    const bool few = E == 1 ? R <= FEW_MAX_DENSE_ROWS : R <= E * FEW_MAX_MEAN_ROWS;
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
