// situ_dispatch.cu — tokens sorted by expert and back (include/situ_moe.h): the row plan, the copy of
// tokens to their rows, the weighted sum of a token's rows and its gradient.
//
// Everything here is bound by HBM (or, for a decoding step's few tokens, by launch and load latency):
// a row is touched once in each pass and nothing of size T·K·D is kept beside the tensors themselves.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/situ_moe.h"
#include "situ_device.cuh"
#include "situ_host.h"

namespace {

using namespace situ;
using namespace situ_host;

constexpr uint32_t FULL = 0xffffffffu;

// ---------------------------------------------------------------------------
// the row plan: a stable counting sort of the T·K expert ids
// ---------------------------------------------------------------------------
// A block owns a contiguous chunk of the ids, a warp a contiguous piece of the chunk, 32 ids a step.
// With every warp's count of every expert known, the prefix over (expert, block, warp) gives each warp
// its first row of each expert; walking its ids again in order, an id's place among the equal ones of
// its step (match) plus the warp's running count is its row. No atomics order anything, so the sort is
// stable and the same every time. Up to PLAN_ONE ids one block does it in one launch; above that a first
// launch writes the blocks' counts [block][expert] and every block of the second one sums what it needs
// (at most PLAN_BLOCKS·E counts, from L2). Measured: see plan_blocks().

constexpr int PLAN_WARPS = 32;
constexpr int PLAN_THREADS = PLAN_WARPS * 32;
constexpr int64_t PLAN_ONE = 4096;           // ids that one block sorts alone
constexpr int64_t PLAN_CHUNK = 2048;         // ids per block above that, until there are PLAN_BLOCKS (262144 ids:
                                             // 17 us; 4096 19 us, 8192 25 us)
constexpr int64_t PLAN_BLOCKS = 152;         // one block per SM: the counts take 132 KB of its shared memory

int64_t plan_blocks(int64_t n) {
    if (n <= PLAN_ONE) return 1;
    const int64_t b = (n + PLAN_CHUNK - 1) / PLAN_CHUNK;
    return b < PLAN_BLOCKS ? b : PLAN_BLOCKS;
}

// The lanes whose id equals this lane's, from one ballot per bit: some 30 instructions whatever the ids are
// (__match_any_sync takes longer the more distinct ids there are: 262144 ids of 896 experts 31 us instead of 15).
__device__ __forceinline__ uint32_t peers_of(uint32_t id, int bits) {
    uint32_t peers = FULL;
    for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(FULL, id >> b & 1u);
        peers &= id >> b & 1u ? set : ~set;
    }
    return peers;
}

__global__ void __launch_bounds__(PLAN_THREADS)
    plan_count_kernel(const int32_t* __restrict__ ids, int* __restrict__ counts, int64_t n, int E, int64_t chunk) {
    __shared__ int hist[SITU_MAX_EXPERTS];
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int64_t b = blockIdx.x * chunk, en = min(n, b + chunk);
    for (int64_t i = b + threadIdx.x; i < en; i += blockDim.x) {
        const int id = ids[i];
        if ((uint32_t)id < (uint32_t)E) atomicAdd(&hist[id], 1);   // a count: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

// counts: [gridDim.x][E] of the first launch, or NULL with one block. `used`: warps that sort (all of them, or
// fewer for few ids); bits: of an expert's number, E (no expert) included.
__global__ void __launch_bounds__(PLAN_THREADS)
    plan_rows_kernel(const int32_t* __restrict__ ids, const float* __restrict__ p, const int* __restrict__ counts,
                     int64_t* __restrict__ offsets, int32_t* __restrict__ row_of, int32_t* __restrict__ src,
                     float* __restrict__ p_rows, int64_t n, int E, int64_t chunk, int used, int bits) {
    extern __shared__ int cnt[];                 // [used][E]: counts, then each warp's next row of each expert
    __shared__ int s_warp[PLAN_WARPS];
    __shared__ int s_total;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int i = threadIdx.x; i < used * E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    // this warp's piece, whole steps of 32 ids
    const int64_t cb = blockIdx.x * chunk, ce = min(n, cb + chunk);
    const int64_t piece = ((chunk + used - 1) / used + 31) / 32 * 32;
    const int64_t b = warp < used ? min(ce, cb + warp * piece) : ce, en = min(ce, b + piece);
    int* mine = cnt + warp * E;
    for (int64_t i = b; i < en; i += 32) {
        const uint32_t id = i + lane < en ? min((uint32_t)ids[i + lane], (uint32_t)E) : (uint32_t)E;
        const uint32_t peers = peers_of(id, bits);
        if (id < (uint32_t)E && lane == __ffs(peers) - 1) mine[id] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    // expert e (one thread each, E <= 1024 threads): rows of all blocks, rows before this block
    int all = 0, before = 0;
    const int e = threadIdx.x;
    if (e < E) {
        int here = 0;
        for (int w = 0; w < used; ++w) here += cnt[w * E + e];
        if (counts) {
            const int nb = (int)gridDim.x;
#pragma unroll 8
            for (int k = 0; k < nb; ++k) {
                const int c = counts[(int64_t)k * E + e];
                all += c;
                before += k < (int)blockIdx.x ? c : 0;
            }
        } else {
            all = here;
        }
    }
    int incl = all;                              // inclusive prefix over the experts
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = lane < warps ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, v, o);
            if (lane >= o) v += u;
        }
        if (lane < warps) s_warp[lane] = v;
    }
    __syncthreads();
    if (warp > 0) incl += s_warp[warp - 1];
    if (threadIdx.x == blockDim.x - 1) s_total = incl;
    if (e < E) {
        if (blockIdx.x == 0) {
            if (e == 0) offsets[0] = 0;
            offsets[e + 1] = incl;
        }
        int row = incl - all + before;
        for (int w = 0; w < used; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = row;
            row += c;
        }
    }
    __syncthreads();
    for (int64_t i = b; i < en; i += 32) {
        const bool in = i + lane < en;
        const uint32_t id = in ? min((uint32_t)ids[i + lane], (uint32_t)E) : (uint32_t)E;
        const uint32_t peers = peers_of(id, bits);
        const bool live = id < (uint32_t)E;
        int row = -1;
        if (live) row = mine[id] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (live && lane == __ffs(peers) - 1) mine[id] += __popc(peers);
        __syncwarp();
        if (in) row_of[i + lane] = row;
        if (live) {
            src[row] = (int32_t)(i + lane);
            if (p_rows) p_rows[row] = p[i + lane];
        }
    }
    // rows that no id has
    for (int64_t r = s_total + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < n; r += (int64_t)gridDim.x * blockDim.x) {
        src[r] = -1;
        if (p_rows) p_rows[r] = 0.0f;
    }
}

// ---------------------------------------------------------------------------
// dispatch, combine and its gradient
// ---------------------------------------------------------------------------

// W elements of a row, as fp32: one 16-byte vector, or one element (W = 1).
template <bool BF16, int W>
struct Elems {
    static constexpr int WORDS = W == 1 ? 1 : 4;
    uint32_t w[WORDS];

    __device__ __forceinline__ void load(const void* base, int64_t at) {
        if constexpr (W == 1) {
            if constexpr (BF16) w[0] = (uint32_t)((const uint16_t*)base)[at];
            else w[0] = ((const uint32_t*)base)[at];
        } else {
            const char* p = (const char*)base + at * (BF16 ? 2 : 4);
            const Vec<4> v = ld_stream<4, false>((const Vec<4>*)p);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = v.w[i];
        }
    }
    // read again soon by other warps or iterations
    __device__ __forceinline__ void load_cached(const void* base, int64_t at) {
        if constexpr (W == 1) {
            load(base, at);
        } else {
            const uint4 v = *(const uint4*)((const char*)base + at * (BF16 ? 2 : 4));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        }
    }
    __device__ __forceinline__ void store(void* base, int64_t at) const {
        if constexpr (W == 1) {
            if constexpr (BF16) ((uint16_t*)base)[at] = (uint16_t)w[0];
            else ((uint32_t*)base)[at] = w[0];
        } else {
            Vec<4> v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v.w[i] = w[i];
            st_stream<4>((Vec<4>*)((char*)base + at * (BF16 ? 2 : 4)), v);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void get(float (&f)[W]) const {
        if constexpr (W == 1) {
            f[0] = BF16 ? bf16_to_f32((uint16_t)w[0]) : __uint_as_float(w[0]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16) {
                    f[2 * i] = bf16_lo(w[i]);
                    f[2 * i + 1] = bf16_hi(w[i]);
                } else {
                    f[i] = __uint_as_float(w[i]);
                }
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[W]) {
        if constexpr (W == 1) {
            w[0] = BF16 ? (uint32_t)f32_to_bf16(f[0]) : __float_as_uint(f[0]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
                else w[i] = __float_as_uint(f[i]);
            }
        }
    }
};

// Rows offsets[E] .. R-1 of h [R, D] belong to no token: zeros, by all threads of the grid. (Clamped:
// malformed offsets cannot reach outside h.)
template <bool BF16, int W>
__device__ __forceinline__ void zero_tail(void* h, const int64_t* offsets, int64_t E, int64_t R, int64_t D) {
    int64_t r0 = offsets[E];
    r0 = r0 < 0 ? 0 : r0;
    if (r0 >= R) return;
    const int64_t n = (R - r0) * (D / W);
    Elems<BF16, W> z;
    z.zero();
    const int64_t grid = (int64_t)gridDim.x * gridDim.y;
    for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += grid * blockDim.x)
        z.store(h, r0 * D + i * W);
}

constexpr int COPY_WARPS = 4;
constexpr int DU = 2;                        // vectors per lane of one dispatch unit

// One warp takes 32·DU vectors of a token's row, loaded once, and stores them to the token's K rows
// (blockIdx.y splits the K rows where there are few tokens): x is read once, h written once.
template <bool BF16, int W, bool WEIGHTED>
__global__ void __launch_bounds__(COPY_WARPS * 32)
    dispatch_kernel(const void* __restrict__ x, const int32_t* __restrict__ row_of, const int64_t* __restrict__ offsets,
                    int64_t E, const float* __restrict__ weights, void* __restrict__ h, int64_t T, int K, int64_t R,
                    int64_t D, int64_t per_row, int kstep) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * COPY_WARPS + (threadIdx.x >> 5);
    const int64_t t = unit / per_row;
    if (t < T) {
        const int64_t c0 = (unit - t * per_row) * (32 * DU) + lane, nv = D / W;
        Elems<BF16, W> v[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u)
            if (c0 + 32 * u < nv) v[u].load(x, t * D + (c0 + 32 * u) * W);
        const int k1 = min(K, ((int)blockIdx.y + 1) * kstep);
        for (int k = (int)blockIdx.y * kstep; k < k1; ++k) {
            const int64_t r = row_of[t * K + k];
            if (r < 0 || r >= R) continue;
            const float wt = WEIGHTED ? weights[t * K + k] : 1.0f;
#pragma unroll
            for (int u = 0; u < DU; ++u) {
                if (c0 + 32 * u >= nv) continue;
                if constexpr (WEIGHTED) {
                    float f[W];
                    v[u].get(f);
#pragma unroll
                    for (int i = 0; i < W; ++i) f[i] *= wt;
                    Elems<BF16, W> o;
                    o.set(f);
                    o.store(h, r * D + (c0 + 32 * u) * W);
                } else {
                    v[u].store(h, r * D + (c0 + 32 * u) * W);
                }
            }
        }
    }
    zero_tail<BF16, W>(h, offsets, E, R, D);
}

constexpr int KB = 8;                        // rows in flight per lane

// One warp takes 32 vectors of a token's output: lane l reads the token's row numbers and weights of
// places l, l + 32, .. once, and KB rows' vectors are loaded before they are added (k ascending).
template <bool BF16, int W>
__global__ void __launch_bounds__(COPY_WARPS * 32)
    combine_kernel(const void* __restrict__ o, const int32_t* __restrict__ row_of, const float* __restrict__ weights,
                   const void* residual, void* y, int64_t T, int K, int64_t R, int64_t D, int64_t per_row) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * COPY_WARPS + (threadIdx.x >> 5);
    const int64_t t = unit / per_row;
    if (t >= T) return;
    const int64_t c = (unit - t * per_row) * 32 + lane;
    const bool in = c < D / W;
    float acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.0f;
    for (int kb = 0; kb < K; kb += 32) {
        int my_row = -1;
        float my_w = 0.0f;
        if (kb + lane < K) {
            my_row = row_of[t * K + kb + lane];
            my_w = weights ? weights[t * K + kb + lane] : 1.0f;
            if (my_row >= R) my_row = -1;
        }
        const int kn = min(32, K - kb);
        for (int k = 0; k < kn; k += KB) {
            Elems<BF16, W> v[KB];
            int row[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                row[j] = __shfl_sync(FULL, my_row, (k + j) & 31);
                if (k + j >= kn) row[j] = -1;
                if (row[j] >= 0 && in) v[j].load(o, (int64_t)row[j] * D + c * W);
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float wt = __shfl_sync(FULL, my_w, (k + j) & 31);
                if (row[j] < 0 || !in) continue;
                float f[W];
                v[j].get(f);
#pragma unroll
                for (int i = 0; i < W; ++i) acc[i] = fmaf(wt, f[i], acc[i]);
            }
        }
    }
    if (!in) return;
    if (residual) {
        Elems<BF16, W> v;
        float f[W];
        v.load(residual, t * D + c * W);
        v.get(f);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] += f[i];
    }
    Elems<BF16, W> out;
    out.set(acc);
    out.store(y, t * D + c * W);
}

constexpr int BWD_MAX_WARPS = 4;              // 128 threads: 430 us at 196624 x 3584 (0.96 of the copy rate); 256: 468, 512: 564

// One block takes a token: every thread holds vectors of dy and walks the token's rows, KB at a time
// (so dy is read K/KB times, all but the first from L1), writing weight·dy and adding dy·o; the KB
// dot products of a thread are summed over the warp, then over the warps in order.
template <bool BF16, int W>
__global__ void __launch_bounds__(BWD_MAX_WARPS * 32)
    combine_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ o, const int32_t* __restrict__ row_of,
                       const float* __restrict__ weights, const int64_t* __restrict__ offsets, int64_t E,
                       void* __restrict__ dout, float* __restrict__ dw, int64_t T, int K, int64_t R, int64_t D) {
    __shared__ float part[BWD_MAX_WARPS][KB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t nv = D / W;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        for (int kb = 0; kb < K; kb += KB) {
            int64_t row[KB];
            float wt[KB], dot[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                row[j] = -1;
                dot[j] = wt[j] = 0.0f;
                if (kb + j < K) {
                    row[j] = row_of[t * K + kb + j];
                    wt[j] = weights[t * K + kb + j];
                    if (row[j] >= R) row[j] = -1;
                }
            }
            for (int64_t c = threadIdx.x; c < nv; c += blockDim.x) {
                Elems<BF16, W> g, v[KB];
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    if (row[j] >= 0) v[j].load(o, row[j] * D + c * W);
                g.load_cached(dy, t * D + c * W);
                float gf[W];
                g.get(gf);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    if (row[j] < 0) continue;
                    float f[W];
                    v[j].get(f);
#pragma unroll
                    for (int i = 0; i < W; ++i) dot[j] = fmaf(gf[i], f[i], dot[j]);
#pragma unroll
                    for (int i = 0; i < W; ++i) f[i] = wt[j] * gf[i];
                    v[j].set(f);
                    v[j].store(dout, row[j] * D + c * W);
                }
            }
#pragma unroll
            for (int j = 0; j < KB; ++j) dot[j] = warp_sum(dot[j]);
            __syncthreads();                 // the previous sums have been read
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < KB; ++j) part[warp][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < KB && kb + (int)threadIdx.x < K) {
                float s = 0.0f;
                for (int w = 0; w < warps; ++w) s += part[w][threadIdx.x];
                dw[t * K + kb + threadIdx.x] = s;
            }
        }
    }
    zero_tail<BF16, W>(dout, offsets, E, R, D);
}

int sm_count(int* n) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return cuda_fail(cudaErrorInvalidDevice);
    LaunchCache& lc = launch_cache();
    std::lock_guard<std::mutex> lock(lc.mu);
    if (lc.sm_count[dev] == 0) {
        int v = 0;
        e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e);
        lc.sm_count[dev] = v;
    }
    *n = lc.sm_count[dev];
    return SITU_GLU_OK;
}

int launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

// Sizes shared by dispatch, combine and its gradient.
int check_rows(int type, int64_t T, int64_t K, int64_t R, int64_t D) {
    if (type != SITU_BF16 && type != SITU_FP32) return SITU_GLU_INVALID_ARG;
    if (T < 0 || K < 1 || K > SITU_MAX_EXPERTS || R < 0 || D < 1 || D > SITU_GLU_MAX_H) return SITU_GLU_INVALID_ARG;
    if (T > INT32_MAX / K || R > INT32_MAX) return SITU_GLU_INVALID_ARG;
    return SITU_GLU_OK;
}

// Blocks of `units` warps of work, or invalid if the grid could not hold them.
int unit_grid(int64_t units, unsigned* grid) {
    const int64_t g = (units + COPY_WARPS - 1) / COPY_WARPS;
    if (g > INT32_MAX) return SITU_GLU_INVALID_ARG;
    *grid = (unsigned)g;
    return SITU_GLU_OK;
}

}  // namespace

extern "C" {

int64_t situ_dispatch_plan_workspace(int64_t T, int64_t K, int64_t E) {
    if (T < 0 || K < 1 || K > SITU_MAX_EXPERTS || T > INT32_MAX / K || E < 1 || E > SITU_MAX_EXPERTS) return 0;
    const int64_t b = plan_blocks(T * K);
    return b > 1 ? b * E * 4 : 0;
}

int situ_dispatch_plan(const int32_t* ids, const float* p, int64_t* expert_offsets, int32_t* row_of, int32_t* src,
                       float* p_rows, void* workspace, int64_t workspace_bytes, int64_t T, int64_t K, int64_t E,
                       cudaStream_t stream) {
    if (T < 0 || K < 1 || K > SITU_MAX_EXPERTS || T > INT32_MAX / K || E < 1 || E > SITU_MAX_EXPERTS)
        return SITU_GLU_INVALID_ARG;
    const int64_t n = T * K, need = situ_dispatch_plan_workspace(T, K, E);
    if (!expert_offsets || !aligned(expert_offsets, 8) || workspace_bytes < need || (need && !workspace))
        return SITU_GLU_INVALID_ARG;
    if (n > 0 && (!ids || !row_of || !src)) return SITU_GLU_INVALID_ARG;
    if (!p != !p_rows) return SITU_GLU_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(p, 4) || !aligned(row_of, 4) || !aligned(src, 4) || !aligned(p_rows, 4) ||
        !aligned(workspace, 4))
        return SITU_GLU_INVALID_ARG;
    const Range in[2] = {range_of(ids, n * 4), range_of(p, p ? n * 4 : 0)};
    const Range out[5] = {range_of(expert_offsets, (E + 1) * 8), range_of(row_of, n * 4), range_of(src, n * 4),
                          range_of(p_rows, p ? n * 4 : 0), range_of(workspace, need)};
    for (int i = 0; i < 5; ++i) {
        for (const Range& r : in)
            if (overlap(out[i], r)) return SITU_GLU_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SITU_GLU_OVERLAP;
    }
    const int64_t blocks = plan_blocks(n);
    const int64_t chunk = blocks > 1 ? (n + blocks - 1) / blocks : n;
    // few ids need few warps; expert e's prefix is thread e's, so at least E threads
    int64_t threads = PLAN_THREADS, used = PLAN_WARPS;
    if (chunk < PLAN_THREADS) {
        used = chunk > 32 ? (chunk + 31) / 32 : 1;
        threads = (E > used * 32 ? E + 31 : used * 32) / 32 * 32;
    }
    int bits = 1;
    while ((E >> bits) != 0) ++bits;
    const size_t smem = (size_t)used * E * 4;
    cudaError_t ce = cudaFuncSetAttribute((const void*)plan_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          PLAN_WARPS * SITU_MAX_EXPERTS * 4);
    if (ce != cudaSuccess) return cuda_fail(ce);
    if (blocks > 1) {
        plan_count_kernel<<<(unsigned)blocks, PLAN_THREADS, 0, stream>>>(ids, (int*)workspace, n, (int)E, chunk);
        const int st = launched();
        if (st != SITU_GLU_OK) return st;
    }
    plan_rows_kernel<<<(unsigned)blocks, (unsigned)threads, smem, stream>>>(
        ids, p, blocks > 1 ? (const int*)workspace : nullptr, expert_offsets, row_of, src, p_rows, n, (int)E, chunk, (int)used, bits);
    return launched();
}

int situ_dispatch(const void* x, int type, const int32_t* row_of, const int64_t* expert_offsets, int64_t E,
                  const float* weights, void* h, int64_t T, int64_t K, int64_t R, int64_t D, cudaStream_t stream) {
    int st = check_rows(type, T, K, R, D);
    if (st != SITU_GLU_OK) return st;
    if (E < 1 || E > SITU_MAX_EXPERTS) return SITU_GLU_INVALID_ARG;
    if (R == 0) return SITU_GLU_OK;
    const int64_t sz = type == SITU_BF16 ? 2 : 4;
    if (!h || !expert_offsets || (T > 0 && (!x || !row_of))) return SITU_GLU_INVALID_ARG;
    if (!aligned(x, (uintptr_t)sz) || !aligned(h, (uintptr_t)sz) || !aligned(row_of, 4) || !aligned(expert_offsets, 8) ||
        !aligned(weights, 4))
        return SITU_GLU_INVALID_ARG;
    const Range rh = range_of(h, R * D * sz);
    if (overlap(rh, range_of(x, T * D * sz)) || overlap(rh, range_of(row_of, T * K * 4)) ||
        overlap(rh, range_of(expert_offsets, (E + 1) * 8)) || (weights && overlap(rh, range_of(weights, T * K * 4))))
        return SITU_GLU_OVERLAP;
    const bool vec = aligned(x, 16) && aligned(h, 16) && D * sz % 16 == 0;
    const int W = vec ? (int)(16 / sz) : 1;
    const int64_t per_row = (D / W + 32 * DU - 1) / (32 * DU);
    unsigned grid = 1;
    if (T > 0 && (st = unit_grid(T * per_row, &grid)) != SITU_GLU_OK) return st;
    // few tokens: the K rows of a token are shared out over more warps
    const int kstep = T * per_row >= 4096 ? (int)K : (T * per_row * 4 >= 4096 ? 4 : 1);
    const dim3 g(grid, (unsigned)((K + kstep - 1) / kstep));
#define SITU_DISPATCH(BF, WW, WT)                                                                                    \
    dispatch_kernel<BF, WW, WT><<<g, COPY_WARPS * 32, 0, stream>>>(x, row_of, expert_offsets, E, weights, h, T, (int)K, \
                                                                  R, D, per_row, kstep)
    if (type == SITU_BF16) {
        if (vec) { if (weights) SITU_DISPATCH(true, 8, true); else SITU_DISPATCH(true, 8, false); }
        else     { if (weights) SITU_DISPATCH(true, 1, true); else SITU_DISPATCH(true, 1, false); }
    } else {
        if (vec) { if (weights) SITU_DISPATCH(false, 4, true); else SITU_DISPATCH(false, 4, false); }
        else     { if (weights) SITU_DISPATCH(false, 1, true); else SITU_DISPATCH(false, 1, false); }
    }
#undef SITU_DISPATCH
    return launched();
}

int situ_combine(const void* o, int type, const int32_t* row_of, const float* weights, const void* residual, void* y,
                 int64_t T, int64_t K, int64_t R, int64_t D, cudaStream_t stream) {
    int st = check_rows(type, T, K, R, D);
    if (st != SITU_GLU_OK) return st;
    if (T == 0) return SITU_GLU_OK;
    const int64_t sz = type == SITU_BF16 ? 2 : 4;
    if ((!o && R > 0) || !row_of || !y) return SITU_GLU_INVALID_ARG;
    if (!aligned(o, (uintptr_t)sz) || !aligned(residual, (uintptr_t)sz) || !aligned(y, (uintptr_t)sz) ||
        !aligned(row_of, 4) || !aligned(weights, 4))
        return SITU_GLU_INVALID_ARG;
    const Range ry = range_of(y, T * D * sz);
    if (overlap(ry, range_of(o, R * D * sz)) || overlap(ry, range_of(row_of, T * K * 4)) ||
        (weights && overlap(ry, range_of(weights, T * K * 4))) ||
        (residual && residual != y && overlap(ry, range_of(residual, T * D * sz))))
        return SITU_GLU_OVERLAP;
    const bool vec = aligned(o, 16) && aligned(y, 16) && aligned(residual, 16) && D * sz % 16 == 0;
    const int W = vec ? (int)(16 / sz) : 1;
    const int64_t per_row = (D / W + 31) / 32;
    unsigned grid = 1;
    if ((st = unit_grid(T * per_row, &grid)) != SITU_GLU_OK) return st;
    auto kernel = type == SITU_BF16 ? (vec ? combine_kernel<true, 8> : combine_kernel<true, 1>)
                                    : (vec ? combine_kernel<false, 4> : combine_kernel<false, 1>);
    kernel<<<grid, COPY_WARPS * 32, 0, stream>>>(o, row_of, weights, residual, y, T, (int)K, R, D, per_row);
    return launched();
}

int situ_combine_bwd(const void* dy, const void* o, int type, const int32_t* row_of, const float* weights,
                     const int64_t* expert_offsets, int64_t E, void* dout_rows, float* dweights, int64_t T, int64_t K,
                     int64_t R, int64_t D, cudaStream_t stream) {
    int st = check_rows(type, T, K, R, D);
    if (st != SITU_GLU_OK) return st;
    if (E < 1 || E > SITU_MAX_EXPERTS) return SITU_GLU_INVALID_ARG;
    if (T == 0 && R == 0) return SITU_GLU_OK;
    const int64_t sz = type == SITU_BF16 ? 2 : 4;
    if (!expert_offsets || (T > 0 && (!dy || !row_of || !weights || !dweights)) || (R > 0 && (!o || !dout_rows)))
        return SITU_GLU_INVALID_ARG;
    if (!aligned(dy, (uintptr_t)sz) || !aligned(o, (uintptr_t)sz) || !aligned(dout_rows, (uintptr_t)sz) ||
        !aligned(row_of, 4) || !aligned(weights, 4) || !aligned(dweights, 4) || !aligned(expert_offsets, 8))
        return SITU_GLU_INVALID_ARG;
    const Range rd = range_of(dout_rows, R * D * sz), rw = range_of(dweights, T * K * 4);
    for (const Range& in : {range_of(dy, T * D * sz), range_of(o, R * D * sz), range_of(row_of, T * K * 4),
                            range_of(weights, T * K * 4), range_of(expert_offsets, (E + 1) * 8)})
        if (overlap(rd, in) || overlap(rw, in)) return SITU_GLU_OVERLAP;
    if (overlap(rd, rw)) return SITU_GLU_OVERLAP;
    int sms = 0;
    if ((st = sm_count(&sms)) != SITU_GLU_OK) return st;
    const bool vec = aligned(dy, 16) && aligned(o, 16) && aligned(dout_rows, 16) && D * sz % 16 == 0;
    const int W = vec ? (int)(16 / sz) : 1;
    // threads: the row's vectors spread evenly over the fewest passes of at most 128 threads
    const int64_t nv = D / W, passes = (nv + BWD_MAX_WARPS * 32 - 1) / (BWD_MAX_WARPS * 32);
    const int threads = (int)(((nv + passes - 1) / passes + 31) / 32 * 32);
    const int64_t most = (int64_t)sms * 64;
    const unsigned grid = (unsigned)(T < 1 ? sms : (T < most ? T : most));
    auto kernel = type == SITU_BF16 ? (vec ? combine_bwd_kernel<true, 8> : combine_bwd_kernel<true, 1>)
                                    : (vec ? combine_bwd_kernel<false, 4> : combine_bwd_kernel<false, 1>);
    kernel<<<grid, threads, 0, stream>>>(dy, o, row_of, weights, expert_offsets, E, dout_rows, dweights, T, (int)K, R, D);
    return launched();
}

}  // extern "C"
