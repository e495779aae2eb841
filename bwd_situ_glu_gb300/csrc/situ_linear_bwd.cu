// situ_linear_bwd.cu — the linear operator's weight and bias gradients, and the step back through its
// activation (include/situ_moe.h). The input gradient is a product like the forward: situ_linear.cu.
//
//   dz = dout·act'(z)                        elementwise, one pass over dout (and the saved z), which also
//   db_e = Σ_{r in e} dz[r]                  sums the unrounded dz: HBM-bound
//   dW_e = Σ_{r in e} dz[r]ᵀ·a[r]            a product per expert that contracts over its rows: tensor cores
#include <cuda.h>
#include <cuda_runtime.h>
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

// ---------------------------------------------------------------- dz and the bias gradient

// Bias sums of 16384 rows x 3584: 22 us with the second kernel (117 MB; 17.5 us at the copy rate).
//
// Rows are cut into pieces of piece_rows() rows of one expert; a block takes a piece's 256 columns at a time
// (8 per lane, its warps take rows in turn), adds its warps' sums in order and leaves them in
// part[piece][column]; the second kernel adds an expert's pieces, every SUM_CHAINS-th in a chain of its own and the chains
// in order. No result depends on timing.
constexpr int BIAS_WARPS = 8;
constexpr int BIAS_COLS = 256;
constexpr int MIN_PIECE = 16, MAX_PIECE = 128, MANY_PIECES = 2048;
constexpr int SUM_CHAINS = 8;
constexpr int64_t SPLIT_PIECES = 16;         // pieces of an expert, on average, from which a chain is a warp's

// 128 rows, or fewer (two a warp at least, 64 pieces of an expert at most) until there are some four blocks an SM:
// 461 x 1088 through silu took 28.9 us with 128. Above MANY_PIECES they grow with the root of the rows: a chain of fp32
// additions is at most 2·sqrt(R) long (one of R/128 lost 0.4 % of the sum of 2^25 equal values), and
// the walk over them is short (2^20 x 3584: 1.06 ms in all, 1.12 at the copy rate; pieces of 128 rows 2.24).
int64_t piece_rows(int64_t R, int64_t N, int64_t E) {
    int64_t piece = MAX_PIECE;
    while (piece > MIN_PIECE && (R / piece + E) * ((N + BIAS_COLS - 1) / BIAS_COLS) < 600 && R / E / piece < 32) piece /= 2;
    while (R / piece > MANY_PIECES && R / piece > piece) piece *= 2;
    return piece;
}

int64_t max_pieces(int64_t R, int64_t N, int64_t E) { return R / piece_rows(R, N, E) + E; }

template <int ACT>
__global__ void __launch_bounds__(BIAS_WARPS * 32)
    act_bwd_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ pre,
                   const int64_t* __restrict__ offsets, uint16_t* __restrict__ dz, float* __restrict__ part, int E,
                   int64_t R, int64_t N, int piece) {
    __shared__ int start[MAX_EXPERTS + 1];
    __shared__ float sums[BIAS_WARPS][BIAS_COLS + 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) start[0] = 0;
    const bool orderly = each_expert(offsets, E, R, [&](int e, int64_t b, int64_t en) {
        start[e + 1] = (int)((en - b + piece - 1) / piece);
    });
    if (!orderly) drop_overlapping(offsets, E, R, start + 1, nullptr);
    if (warp == 0) prefix_in_place(start, E, lane);
    __syncthreads();
    const int64_t cb = (N + BIAS_COLS - 1) / BIAS_COLS, items = (int64_t)start[E] * cb;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int t = (int)(it / cb);
        const int64_t col = (it - (int64_t)t * cb) * BIAS_COLS + lane * 8;
        int lo = 0, hi = E - 1;              // last e with start[e] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= t) lo = mid; else hi = mid - 1;
        }
        int64_t b, en;
        expert_range(offsets, lo, R, b, en);
        const int64_t r0 = b + (int64_t)(t - start[lo]) * piece;
        const int64_t r1 = min(en, r0 + piece);
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = 0.0f;
        if (col < N) {                       // N % 8 == 0: whole vectors
#pragma unroll 8
            for (int64_t r = r0 + warp; r < r1; r += BIAS_WARPS) {
                const Vec<4> g = ld_stream<4, true>((const Vec<4>*)(dout + r * N + col));
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = bf16_lo(g.w[i]);
                    f[2 * i + 1] = bf16_hi(g.w[i]);
                }
                if constexpr (ACT != SITU_ACT_NONE) {
                    const Vec<4> z = ld_stream<4, true>((const Vec<4>*)(pre + r * N + col));
                    Vec<4> o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[2 * i] *= act_grad<ACT>(bf16_lo(z.w[i]));
                        f[2 * i + 1] *= act_grad<ACT>(bf16_hi(z.w[i]));
                        o.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
                    }
                    st_stream<4>((Vec<4>*)(dz + r * N + col), o);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += f[i];
            }
        }
        if (part) {                          // uniform over the grid
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = s[i];
            __syncthreads();
            const int64_t c = (it - (int64_t)t * cb) * BIAS_COLS + threadIdx.x;
            if (c < N) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < BIAS_WARPS; ++w) v += sums[w][threadIdx.x];
                part[(int64_t)t * N + c] = v;
            }
            __syncthreads();
        }
    }
}

// blockIdx.y: expert; blockIdx.x: BIAS_COLS columns, their chains in a thread's registers, or 32 columns, a chain a
// warp (SPLIT, for experts of many pieces: 16384 x 3584 for one weight, 128 pieces, 32.9 us in registers, 21.8 split; 256 experts
// of 1024 x 1024, 8 pieces each, 87.5 and 100.6). The same sums either way.
template <bool SPLIT>
__global__ void __launch_bounds__(BIAS_COLS)
    bias_sum_kernel(const float* __restrict__ part, const int64_t* __restrict__ offsets, float* __restrict__ dbias,
                    int64_t R, int64_t N, int piece) {
    static_assert(SUM_CHAINS == BIAS_COLS / 32, "a chain a warp");
    const int e = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float s_chain[SUM_CHAINS][32];
    __shared__ int s_first[BIAS_COLS / 32];
    __shared__ int s_count[MAX_EXPERTS];
    const bool orderly = each_expert(offsets, (int)gridDim.y, R, [&](int i, int64_t b, int64_t en) {
        s_count[i] = (int)((en - b + piece - 1) / piece);
    });
    if (!orderly) drop_overlapping(offsets, (int)gridDim.y, R, s_count, nullptr);
    int first = 0;                           // pieces of the experts before e
    for (int i = threadIdx.x; i < e; i += blockDim.x) first += s_count[i];
    first = (int)__reduce_add_sync(FULL_MASK, (unsigned)first);
    if (lane == 0) s_first[warp] = first;
    __syncthreads();
    first = 0;
#pragma unroll
    for (int i = 0; i < BIAS_COLS / 32; ++i) first += s_first[i];
    const int64_t n = s_count[e];
    const int64_t c = (int64_t)blockIdx.x * (SPLIT ? 32 : BIAS_COLS) + (SPLIT ? lane : threadIdx.x);
    const float* at = part + first * N + c;
    float v[SUM_CHAINS] = {};
    if constexpr (SPLIT) {
        if (c < N) {
#pragma unroll 8
            for (int64_t i = warp; i < n; i += SUM_CHAINS) v[0] += at[i * N];
        }
        s_chain[warp][lane] = v[0];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int k = 0; k < SUM_CHAINS; ++k) v[k] = s_chain[k][lane];
    } else if (c < N) {
        for (int64_t i = 0; i < n; i += SUM_CHAINS) {
#pragma unroll
            for (int k = 0; k < SUM_CHAINS; ++k)
                if (i + k < n) v[k] += at[(i + k) * N];
        }
    }
    if (c >= N) return;
#pragma unroll
    for (int k = 1; k < SUM_CHAINS; ++k) v[0] += v[k];
    dbias[(int64_t)e * N + c] = v[0];
}

// ---------------------------------------------------------------- the weight gradient

// dW_e [N, K] = dz_eᵀ·a_e on the tensor cores, on pairs of SMs (situ_pair.cuh). A job is a 256 x 256 tile of one
// expert's dW; its contraction runs over the expert's rows, 64 to a ring stage. Both operands are read as they
// are stored, rows apart ("MN-major": per stage and CTA two 64-column boxes of dz and two of a, 128-byte swizzle).
//
// A TMA box cannot end at an expert's last row, so its last stage brings rows of the next expert (or zeros past
// the tensor). Only the 16-row steps that hold rows of the expert are issued, and where the last of them is
// partial both CTAs first zero the rows past the end, in both operands (generic-proxy writes, the proxy fence, an
// arrival at the leader's tail_ready), so nothing of another expert enters, NaN included. Such a stage's
// loads count at the CTA's own tail_full barrier of that stage, since each CTA must see its own (one barrier a stage:
// experts of a few rows have several ragged stages in the ring).
//
// The tensor cores cut each step's fp32 sum towards zero, an error that grows with the steps (measured
// against float64 at 2048 x 2048: 5e-7 of the norm after 512 rows, 4.4e-6 after 4096, 1.9e-5 after
// 16384). dW feeds an fp32 optimizer, so an accumulator takes CHUNK_BLOCKS stages (512 rows; up to three more
// where that finishes the job) and the epilogue's threads add the chunks in registers, rounded to nearest, while the tensor cores
// fill the other accumulator. Where the tiles of dW cannot fill the SMs, the rows are cut into `splits` pieces
// whose sums (fp32, in the workspace) a second kernel adds in order.
constexpr int CHUNK_BLOCKS = 8, CHUNK_MORE = 3;
constexpr int EPW = 2;
constexpr int NUM_EPI_WARPS = 4 * EPW;
constexpr int TAIL_WARP = 2 + NUM_EPI_WARPS;
constexpr int NUM_THREADS = (3 + NUM_EPI_WARPS) * 32;   // TMA, MMA, epilogue, tails
constexpr int TILE = 256;
constexpr int STAGE_TILE = 32 * 128;         // 32 rows x 128 bytes of dW
constexpr int SBYTES = PA_BYTES + PB_BYTES;
constexpr int STAGES_W = 5;
static_assert(STAGES_W <= PSTAGES, "ring barriers");

struct WPlan {
    int begin[MAX_EXPERTS];                  // first row and rows of each expert
    int rows[MAX_EXPERTS];
};
constexpr int SMEM_BYTES = 1024 + STAGES_W * SBYTES + NUM_EPI_WARPS * STAGE_TILE + (int)sizeof(PairBars) + (int)sizeof(WPlan);
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

struct WJob {
    int mt, nt, plane;
    int row0, rows;                          // rows to contract over
};

// A job of kbs stages: whether its chunk ends with stage kb, in_chunk stages after the chunk's first, and its chunks.
__device__ __forceinline__ bool chunk_ends_at(int kb, int in_chunk, int kbs) {
    return kb + 1 == kbs || (in_chunk + 1 >= CHUNK_BLOCKS && kbs - kb - 1 > CHUNK_MORE);
}
__device__ __forceinline__ int chunk_count(int kbs) {
    return kbs <= CHUNK_BLOCKS + CHUNK_MORE ? (kbs > 0) : 1 + (kbs - CHUNK_MORE - 1) / CHUNK_BLOCKS;
}

// The order of a job's stages. Zeroing a ragged last block takes some 0.5 us after it has landed; where a job has three
// blocks or more it is therefore loaded third from last and used last, while the two after it are worked off.
// i-th load -> block; i-th use -> which load it uses. (Ragged experts of ~1024 rows: 297 -> 283 us.)
__device__ __forceinline__ int loaded_block(int i, int kbs, bool early) {
    return early && i >= kbs - 3 ? (i == kbs - 3 ? kbs - 1 : i - 1) : i;
}
__device__ __forceinline__ int used_load(int i, int kbs, bool early) {
    return early && i >= kbs - 3 ? (i == kbs - 1 ? kbs - 3 : i + 1) : i;
}

// Job j: experts, then pieces of their rows, then tiles of dW. 32-bit: the host bounds their number.
__device__ __forceinline__ WJob wgrad_job(int j, const WPlan& plan, int E, int MT, int NT, int splits) {
    WJob w;
    const int jm = j / NT;
    w.nt = j - jm * NT;
    const int js = jm / MT;
    w.mt = jm - js * MT;
    const int e = js / splits, s = js - e * splits;
    w.plane = s * E + e;
    const int rows = plan.rows[e];
    const int piece = ((rows + BK - 1) / BK + splits - 1) / splits * BK;
    w.row0 = plan.begin[e] + min(rows, s * piece);
    w.rows = min(rows, (s + 1) * piece) - min(rows, s * piece);
    return w;
}

// OUT_FP32: dW (or a partial sum) in fp32, else bf16.
template <bool OUT_FP32>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap map_dz, const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_dw, const int64_t* __restrict__ offsets,
                 int* __restrict__ status, int E, int64_t R, int64_t N, int64_t K, int MT, int NT, int splits) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* staging = ring + STAGES_W * SBYTES;
    PairBars* bars = (PairBars*)(staging + NUM_EPI_WARPS * STAGE_TILE);
    WPlan& plan = *(WPlan*)(bars + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int jobs = E * splits * MT * NT;
    const int j0 = blockIdx.x >> 1, jstep = gridDim.x >> 1;

    const bool orderly = each_expert(offsets, E, R, [&](int e, int64_t b, int64_t en) {
        plan.begin[e] = (int)b;
        plan.rows[e] = (int)(en - b);
    });
    if (!orderly) drop_overlapping(offsets, E, R, plan.rows, nullptr);
    const uint32_t tmem = pair_setup(bars, NUM_EPI_WARPS);

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs; the warp converged, one lane issues)
        const bool elected = elect_one();
        int stage = 0;
        uint32_t phase = 0, pending = 0, pend_par = 0;
        uint32_t tail_used = 0, tail_next = 0;                   // bit s: stage s held a ragged stage; the next one's parity
        const uint64_t pol = make_policy<L2Hint::normal>();
        bool ok = true;
        WJob next = wgrad_job(j0, plan, E, MT, NT, splits);
        for (int j = j0; ok && j < jobs; j += jstep) {
            const WJob w = next;
            const int kbs = (w.rows + BK - 1) / BK;
            const bool ragged = (w.rows & (UK - 1)) != 0, early = ragged && kbs >= 3;
            const int ca = w.mt * TILE + rank * 128, cb = w.nt * TILE + rank * 128;
            if (kbs == 0 && j + jstep < jobs) next = wgrad_job(j + jstep, plan, E, MT, NT, splits);
            for (int i = 0; i < kbs; ++i) {
                const int kb = loaded_block(i, kbs, early);
                if (!pair_wait(&bars->empty[stage], phase ^ 1, &bars->abort, status)) { ok = false; break; }
                if (elected) {
                    uint8_t* sa = ring + stage * SBYTES;
                    const int row = w.row0 + kb * BK;
                    uint32_t bar;
                    if (ragged && kb + 1 == kbs) {
                        if (rank == 0) mbar_arrive(&bars->full[stage]);
                        mbar_expect_tx(&bars->tail_full[stage], SBYTES);
                        bar = smem_addr(&bars->tail_full[stage]);
                    } else {
                        if (rank == 0) mbar_expect_tx(&bars->full[stage], 2 * SBYTES);
                        bar = cluster_addr(&bars->full[stage], 0);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        pair_load_2d(sa + h * PBOX_BYTES, &map_dz, ca + 64 * h, row, bar, pol);
                        pair_load_2d(sa + PA_BYTES + h * PBOX_BYTES, &map_a, cb + 64 * h, row, bar, pol);
                    }
                }
                if (ragged && kb + 1 == kbs) {
                    tail_used |= 1u << stage;
                    tail_next ^= 1u << stage;
                }
                pending |= 1u << stage;
                pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES_W) { stage = 0; phase ^= 1; }
                if (i == 0 && j + jstep < jobs) next = wgrad_job(j + jstep, plan, E, MT, NT, splits);   // while these fly
            }
        }
        __syncwarp();
        if (rank == 0) pair_drain(bars, pending, pend_par);
        for (int s = 0; s < STAGES_W; ++s)
            if (tail_used >> s & 1) mbar_drain(&bars->tail_full[s], (tail_next >> s & 1) ^ 1);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader; the warp converged, one lane issues)
        const bool elected = elect_one();
        uint32_t base = 0, tails = 0;                            // loads before this job; bit s: parity of stage s's next ragged use
        int done = 0;
        bool ok = true;
        const uint32_t idesc = pair_idesc(TILE, true, true);
        const uint32_t ring_addr = smem_addr(ring);
        int rows_next = wgrad_job(j0, plan, E, MT, NT, splits).rows;
        for (int j = j0; rank == 0 && ok && j < jobs; j += jstep) {
            const int rows = rows_next;
            const int kbs = (rows + BK - 1) / BK;
            const bool ragged = (rows & (UK - 1)) != 0, early = ragged && kbs >= 3;
            if (kbs == 0 && j + jstep < jobs) rows_next = wgrad_job(j + jstep, plan, E, MT, NT, splits).rows;
            int in_chunk = 0;
            for (int i = 0; i < kbs; ++i) {
                const uint32_t load = base + (uint32_t)used_load(i, kbs, early), stage = load % STAGES_W, phase = load / STAGES_W & 1;
                const bool last = i + 1 == kbs;                  // block kbs - 1, whichever load brought it
                const int steps = last ? (rows - (kbs - 1) * BK + UK - 1) / UK : BK / UK, acc = done & 1;
                const bool chunk_ends = chunk_ends_at(i, in_chunk, kbs);
                if (in_chunk == 0) ok = pair_wait<true>(&bars->tempty[acc], (uint32_t)((done >> 1) & 1) ^ 1, &bars->abort, status);
                if (ok) ok = pair_wait(&bars->full[stage], phase, &bars->abort, status);
                if (ok && last && ragged) {
                    ok = pair_wait<true>(&bars->tail_ready[stage], tails >> stage & 1, &bars->abort, status);
                    tails ^= 1u << stage;
                }
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * 256), sa = ring_addr + stage * SBYTES;
                const uint64_t ad = smem_desc_mn(sa), bd = smem_desc_mn(sa + PA_BYTES);
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < BK / UK; ++kk)         // 16 rows = 2048 bytes further (128 descriptor units)
                        if (kk < steps)
                            pair_mma(d, ad + (uint64_t)(kk * 128), bd + (uint64_t)(kk * 128), idesc,
                                     kk > 0 ? 1u : (uint32_t)in_chunk);
                    pair_commit(&bars->empty[stage]);
                    if (chunk_ends) pair_commit(&bars->tfull[acc]);
                }
                done += chunk_ends;
                in_chunk = chunk_ends ? 0 : in_chunk + 1;
                if (i == 0 && j + jstep < jobs) rows_next = wgrad_job(j + jstep, plan, E, MT, NT, splits).rows;   // while these run
            }
            base += (uint32_t)kbs;
        }
        __syncwarp();
        if (rank == 0 && elected) pair_commit(&bars->mma_done);
    } else if (warp == TAIL_WARP) {
        // ------------------------------------------------ ragged tails (both CTAs): zeroed as soon as they land, while the
        // stages before them are still being worked off (in the MMA warp this cost 1.1 us of every job)
        int stage = 0;
        uint32_t tails = 0;
        bool ok = true;
        for (int j = j0; ok && j < jobs; j += jstep) {
            const int rows = wgrad_job(j, plan, E, MT, NT, splits).rows;
            const int kbs = (rows + BK - 1) / BK;
            const int st = (stage + kbs - (kbs >= 3 ? 3 : 1) + STAGES_W) % STAGES_W;   // where its last block is loaded
            stage = (stage + kbs) % STAGES_W;
            if ((rows & (UK - 1)) == 0) continue;
            ok = pair_wait(&bars->tail_full[st], tails >> st & 1, &bars->abort, status);
            if (!ok) break;
            tails ^= 1u << st;
            const int valid = rows - (kbs - 1) * BK;
            const int n16 = (UK - (valid & (UK - 1))) * 8;                   // 16-byte pieces per box, to the step's end
            uint8_t* sa = ring + st * SBYTES;
            for (int i = lane; i < n16 * (SBYTES / PBOX_BYTES); i += 32) {
                const int box = i / n16;
                st_shared_v4(sa + box * PBOX_BYTES + valid * 128 + (i - box * n16) * 16, 0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(cluster_addr(&bars->tail_ready[st], 0));
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs): a lane holds one row of dW
        const int quad = warp & 3;
        const int slot = (warp - 2) >> 2;
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        uint8_t* stage = staging + (warp - 2) * STAGE_TILE;
        constexpr int COLS = TILE / EPW;             // columns of this warp
        constexpr int CW = OUT_FP32 ? 32 : 64;       // columns per 128-byte staged row
        bool stores_pending = false;
        int done = 0;
        for (int j = j0; j < jobs; j += jstep) {
            const WJob w = wgrad_job(j, plan, E, MT, NT, splits);
            const int chunks = chunk_count((w.rows + BK - 1) / BK);
            bool ok = true;
            float sum[COLS];
#pragma unroll
            for (int i = 0; i < COLS; ++i) sum[i] = 0.0f;
            for (int ch = 0; ch < chunks; ++ch, ++done) {
                const int acc = done & 1;
                ok = pair_wait_epilogue(&bars->tfull[acc], (uint32_t)((done >> 1) & 1), bars, status, NUM_EPI_WARPS);
                if (ok) {
#pragma unroll
                    for (int h = 0; h < COLS; h += 16) {
                        float v[16];
                        tc_ld<16>(tmem + t_lane + (uint32_t)(acc * 256 + slot * COLS + h), v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[h + i] += v[i];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&bars->tempty[acc], 0));
            }
            const int n0 = w.mt * TILE + rank * 128 + quad * 32;
#pragma unroll
            for (int c = 0; c < COLS; c += CW) {
                const int col = w.nt * TILE + slot * COLS + c;
                if (!ok || n0 >= N || col >= K) continue;      // uniform over the warp
                if (stores_pending) {
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint8_t* at = stage + lane * 128 + ((q ^ (lane & 7)) << 4);
                    if constexpr (OUT_FP32) {
                        st_shared_v4(at, __float_as_uint(sum[c + 4 * q]), __float_as_uint(sum[c + 4 * q + 1]),
                                     __float_as_uint(sum[c + 4 * q + 2]), __float_as_uint(sum[c + 4 * q + 3]));
                    } else {
                        uint32_t p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = pack_bf16x2(sum[c + 8 * q + 2 * i], sum[c + 8 * q + 2 * i + 1]);
                        st_shared_v4(at, p[0], p[1], p[2], p[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&map_dw, col, n0, w.plane, stage);
                    bulk_commit();
                }
                stores_pending = true;
            }
        }
        if (lane == 0 && stores_pending) bulk_wait_all();
    }
    pair_teardown(tmem, bars);
}

// dw = the sum of `splits` partial sums of n elements each, in order.
template <bool OUT_FP32>
__global__ void __launch_bounds__(256)
    wgrad_sum_kernel(const float* __restrict__ part, void* __restrict__ dw, int64_t n, int splits) {
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * blockDim.x * 4) {
        float4 s = *(const float4*)(part + i);           // n % 4 == 0
        for (int k = 1; k < splits; ++k) {
            const float4 v = *(const float4*)(part + k * n + i);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        if constexpr (OUT_FP32) *(float4*)((float*)dw + i) = s;
        else *(uint2*)((uint16_t*)dw + i) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
}

constexpr int64_t MAX_SPLITS = 16;
constexpr int64_t SPLIT_MIN_ROWS = 256;      // a piece of fewer rows does not pay for its partial sum
constexpr int SM_COUNT = 152;                // what the workspace is sized for: the split must not need a device

// Pieces of the contraction: as many as fill the pairs of SMs with jobs.
int64_t wgrad_splits(int64_t R, int64_t N, int64_t K, int64_t E) {
    const int64_t jobs = E * ((N + TILE - 1) / TILE) * ((K + TILE - 1) / TILE);
    int64_t s = SM_COUNT / 2 / jobs;
    const int64_t most = R / E / SPLIT_MIN_ROWS;
    if (s > most) s = most;
    if (s > MAX_SPLITS) s = MAX_SPLITS;
    return s < 1 ? 1 : s;
}


}  // namespace

extern "C" {

int64_t situ_linear_act_bwd_workspace(int64_t R, int64_t N, int64_t E) {
    if (check_linear(E, (const void*)8, R, N, 8) != SITU_GLU_OK) return 0;
    return max_pieces(R, N, E) * N * 4;
}

int situ_linear_act_bwd(const void* dout, const void* pre, int act, const int64_t* expert_offsets, int64_t E, void* dz,
                        float* dbias, void* workspace, int64_t workspace_bytes, int64_t R, int64_t N,
                        cudaStream_t stream) {
    int st = check_linear(E, expert_offsets, R, N, 8);
    if (st != SITU_GLU_OK) return st;
    if (act < SITU_ACT_NONE || act > SITU_ACT_GELU) return SITU_GLU_INVALID_ARG;
    const bool with_dz = act != SITU_ACT_NONE;
    const int piece = (int)piece_rows(R, N, E);
    const int64_t need = dbias ? situ_linear_act_bwd_workspace(R, N, E) : 0;
    if (R > 0 && (!dout || (with_dz && (!pre || !dz)))) return SITU_GLU_INVALID_ARG;
    if (dbias && (workspace_bytes < need || !workspace)) return SITU_GLU_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(pre, 16) || !aligned(dz, 16) || !aligned(dbias, 4) || !aligned(workspace, 4) ||
        !aligned(expert_offsets, 8))
        return SITU_GLU_INVALID_ARG;
    const Range in[3] = {range_of(dout, R * N * 2), range_of(pre, with_dz ? R * N * 2 : 0),
                         range_of(expert_offsets, expert_offsets ? (E + 1) * 8 : 0)};
    const Range o[3] = {range_of(dz, with_dz ? R * N * 2 : 0), range_of(dbias, dbias ? E * N * 4 : 0),
                        range_of(workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (overlap(o[i], r)) return SITU_GLU_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(o[i], o[j])) return SITU_GLU_OVERLAP;
    }
    if (R > 0 && (with_dz || dbias)) {
        auto kernel = act == SITU_ACT_RELU ? act_bwd_kernel<SITU_ACT_RELU> : act == SITU_ACT_SILU ? act_bwd_kernel<SITU_ACT_SILU>
                      : act == SITU_ACT_GELU ? act_bwd_kernel<SITU_ACT_GELU> : act_bwd_kernel<SITU_ACT_NONE>;
        int grid = 0;
        const int64_t items = max_pieces(R, N, E) * ((N + BIAS_COLS - 1) / BIAS_COLS);
        st = grid_for((const void*)kernel, BIAS_WARPS * 32, items * BIAS_WARPS, &grid);
        if (st != SITU_GLU_OK) return st;
        // several blocks a place: the pieces are short and uneven
        if ((int64_t)grid * 4 < items) grid *= 4; else grid = (int)items;
        kernel<<<grid, BIAS_WARPS * 32, 0, stream>>>((const uint16_t*)dout, (const uint16_t*)pre, expert_offsets,
                                                     (uint16_t*)dz, dbias ? (float*)workspace : nullptr, (int)E, R, N, piece);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e);
    }
    if (dbias) {
        const bool split = R / piece / E >= SPLIT_PIECES;
        const int64_t cols = split ? 32 : BIAS_COLS;
        auto kernel = split ? bias_sum_kernel<true> : bias_sum_kernel<false>;
        kernel<<<dim3((unsigned)((N + cols - 1) / cols), (unsigned)E), BIAS_COLS, 0, stream>>>((const float*)workspace,
                                                                                              expert_offsets, dbias, R, N, piece);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return SITU_GLU_OK;
}

int64_t situ_linear_wgrad_workspace(int64_t R, int64_t N, int64_t K, int64_t E) {
    if (check_linear(E, (const void*)8, R, N, K) != SITU_GLU_OK) return 0;
    const int64_t s = wgrad_splits(R, N, K, E);
    return s > 1 ? s * E * N * K * 4 : 0;
}

int situ_linear_wgrad(const void* dz, const void* a, const int64_t* expert_offsets, int64_t E, void* dw, int dw_type,
                      void* workspace, int64_t workspace_bytes, int* status, int64_t R, int64_t N, int64_t K,
                      cudaStream_t stream) {
    int st = check_linear(E, expert_offsets, R, N, K);
    if (st != SITU_GLU_OK) return st;
    if (dw_type != SITU_BF16 && dw_type != SITU_FP32) return SITU_GLU_INVALID_ARG;
    const int64_t need = situ_linear_wgrad_workspace(R, N, K, E);
    if (!dw || (R > 0 && (!dz || !a)) || workspace_bytes < need || (need && !workspace)) return SITU_GLU_INVALID_ARG;
    if (!aligned(dz, 16) || !aligned(a, 16) || !aligned(dw, 16) || !aligned(workspace, 16) ||
        !aligned(expert_offsets, 8) || !aligned(status, 4))
        return SITU_GLU_INVALID_ARG;
    const int64_t dw_bytes = E * N * K * (dw_type == SITU_FP32 ? 4 : 2);
    const Range in[3] = {range_of(dz, R * N * 2), range_of(a, R * K * 2),
                         range_of(expert_offsets, expert_offsets ? (E + 1) * 8 : 0)};
    const Range o[3] = {range_of(dw, dw_bytes), range_of(workspace, need), range_of(status, status ? 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (overlap(o[i], r)) return SITU_GLU_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(o[i], o[j])) return SITU_GLU_OVERLAP;
    }
    if (R == 0) {
        const cudaError_t e = cudaMemsetAsync(dw, 0, (size_t)dw_bytes, stream);
        return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
    }
    const int64_t splits = wgrad_splits(R, N, K, E);
    const bool fp32 = splits > 1 || dw_type == SITU_FP32;
    const int MT = (int)((N + TILE - 1) / TILE), NT = (int)((K + TILE - 1) / TILE);
    if (E * splits * MT * NT > INT32_MAX / 2) return SITU_GLU_INVALID_ARG;   // the kernel counts jobs in 32 bits
    CUtensorMap map_dz, map_a, map_dw;
    if (!make_map(&map_dz, dz, (uint64_t)R, (uint64_t)N, BK) || !make_map(&map_a, a, (uint64_t)R, (uint64_t)K, BK))
        return cuda_fail(cudaErrorInvalidValue);
    const uint64_t sz = fp32 ? 4 : 2;
    const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)(E * splits)};
    const uint64_t strides[2] = {(uint64_t)K * sz, (uint64_t)K * (uint64_t)N * sz};
    const uint32_t box[3] = {(uint32_t)(128 / sz), 32, 1};
    if (!make_map_any(&map_dw, splits > 1 ? workspace : dw, fp32, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cuda_fail(cudaErrorInvalidValue);
    int sms = 0;
    if ((st = sm_count(&sms)) != SITU_GLU_OK) return st;
    cudaError_t e = launch_pairs(fp32 ? wgrad_kernel<true> : wgrad_kernel<false>, E * splits * MT * NT, NUM_THREADS, SMEM_BYTES,
                                 stream, map_dz, map_a, map_dw, expert_offsets, status, (int)E, R, N, K, MT, NT, (int)splits);
    if (e != cudaSuccess) return cuda_fail(e);
    if (splits > 1) {
        const int64_t n = E * N * K, blocks = (n / 4 + 255) / 256;
        const unsigned grid = (unsigned)(blocks < sms * 8 ? blocks : sms * 8);
        if (dw_type == SITU_FP32) wgrad_sum_kernel<true><<<grid, 256, 0, stream>>>((const float*)workspace, dw, n, (int)splits);
        else wgrad_sum_kernel<false><<<grid, 256, 0, stream>>>((const float*)workspace, dw, n, (int)splits);
        if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e);
    }
    return SITU_GLU_OK;
}

}  // extern "C"
