// situ_route.cu — top-k softmax of the router scores and its gradient (include/situ_moe.h).
//
//   forward   ids = the K largest of s[t, :] (ties: lowest index), p = softmax of them
//   backward  ds[t, id_k] = p_k·(dp_k − Σ_j p_j·dp_j), 0 elsewhere
//
// Both are bound by HBM: the forward reads T·E scores once, the backward writes T·E once; at
// T = 65537, E = 896 in fp32 that is 235 MB, 35 us at the measured copy rate, for each.
//
// Forward, one warp per token: lane i holds the scores i·W .. of each 32·W-wide chunk in registers. The 35 us hold
// some 600 instructions a token, and a full sort, or K rounds of a warp-wide maximum (K·(reduction + rescan of a
// lane's 28 scores) ≈ 1100 at E = 896, K = 16), take more. Instead: the K-th largest of the 32 lane maxima is a
// lower bound of the K-th largest score, so only scores at or above it can be chosen; on random scores about 20
// of 896 are left, one per lane, picked by a bit mask from the row's copy in shared memory. The maxima are ordered by
// a bitonic sort, the candidates by counting the better ones in shared memory: together 47 us at T = 65537 (both by
// sorts 49: 30 dependent shuffles; both by counting 55: bound by issue). Where more than 32 are left (many equal scores, a sorted row), or a score is NaN, K rounds of
// a warp-wide maximum run instead: the same result.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/situ_moe.h"
#include "situ_device.cuh"
#include "situ_host.h"

namespace {

using namespace situ;
using namespace situ_host;

constexpr int WARPS = 4;                     // warps (tokens) per CTA
constexpr uint32_t FULL = 0xffffffffu;

// Order-preserving key: larger score, larger key; -0 and +0 alike, every NaN on top; 0 is below
// every score and marks "no score".
__device__ __forceinline__ uint32_t score_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return (u & 0x7fffffffu) > 0x7f800000u ? FULL : k;
}
constexpr uint32_t KEY_MINUS_INF = 0x007fffffu;

__device__ __forceinline__ float key_score(uint32_t k) {
    if (k == FULL) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// W consecutive scores from global memory as floats; W = 1 or one 16-byte vector.
template <bool BF16, int W>
__device__ __forceinline__ void load_scores(const void* base, int64_t at, float (&v)[W]) {
    if constexpr (W == 1) {
        if constexpr (BF16) v[0] = bf16_to_f32(((const uint16_t*)base)[at]);
        else v[0] = ((const float*)base)[at];
    } else if constexpr (BF16) {
        static_assert(W == 8, "one 16-byte vector");
        const Vec<4> r = ld_stream<4, true>((const Vec<4>*)((const uint16_t*)base + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(r.w[i]);
            v[2 * i + 1] = bf16_hi(r.w[i]);
        }
    } else {
        static_assert(W == 4, "one 16-byte vector");
        const Vec<4> r = ld_stream<4, true>((const Vec<4>*)((const float*)base + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
    }
}

// BF16: score type. W: scores per load. C: loads per lane (32·W·C >= E).
template <bool BF16, int W, int C>
__global__ void __launch_bounds__(WARPS * 32, 10)   // 48 registers: the sort waits on shuffles, so more warps (59 -> 49 us)
    route_topk_kernel(const void* __restrict__ logits, float* __restrict__ p, int32_t* __restrict__ ids, int64_t T,
                      int E, int K) {
    constexpr int CHUNK = 32 * W;             // scores per chunk
    __shared__ alignas(16) uint64_t s_cand[WARPS][32];           // (key, ~index) of the candidates
    __shared__ float s_row[WARPS][C * CHUNK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * WARPS + warp;
    if (t >= T) return;

    float v[C][W];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = c * CHUNK + lane * W;
        if (e < E) {
            load_scores<BF16, W>(logits, t * E + e, v[c]);      // W divides E: whole vectors
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) v[c][i] = -INFINITY;
        }
    }
    float top = -INFINITY;                    // the lane's maximum; NaN if it has one
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(v[c][i]));
            s_row[warp][c * CHUNK + lane * W + i] = v[c][i];
        }
    }
    // the K-th largest lane maximum (bitonic sort, descending over the lanes)
    const uint32_t mine_top = score_key(top);
    s_cand[warp][lane] = 0;
    uint32_t srt = mine_top;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
            const uint32_t other = __shfl_xor_sync(FULL, srt, o);
            const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
            srt = keep_max ? max(srt, other) : min(srt, other);
        }
    }
    const bool nan = __any_sync(FULL, mine_top == FULL);
    // every score above -inf is at or above the lowest finite one
    const float bound = fmaxf(key_score(__shfl_sync(FULL, srt, K - 1)), -3.402823466e38f);

    uint32_t mask = 0;                        // bit c·W + i: v[c][i] is a candidate
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < W; ++i) mask |= v[c][i] >= bound ? 1u << (c * W + i) : 0u;
    const int n = __popc(mask);
    int at = n;                               // inclusive prefix of n over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL, at, o);
        if (lane >= o) at += u;
    }
    const int total = __shfl_sync(FULL, at, 31);

    uint32_t my_key = 0, my_idx = FULL;       // lane k's result: the k-th largest
    if (total <= 32 && !nan) {
        at -= n;
        __syncwarp();                         // the slots are empty
        for (; mask; mask &= mask - 1) {
            const int b = __ffs(mask) - 1;
            const int idx = b / W * CHUNK + lane * W + b % W;
            // this lane's own store; larger is better: by score, then by lower index
            s_cand[warp][at++] = (uint64_t)score_key(s_row[warp][idx]) << 32 | ~(uint32_t)idx;
        }
        __syncwarp();
        // a candidate's place is the number of better ones (they differ in their index); empty slots are 0
        const uint64_t mine = s_cand[warp][lane];
        int place = 0;
        for (int q = 0; q < total; q += 4) {
            const ulonglong2 c0 = *(const ulonglong2*)&s_cand[warp][q], c1 = *(const ulonglong2*)&s_cand[warp][q + 2];
            place += (c0.x > mine) + (c0.y > mine) + (c1.x > mine) + (c1.y > mine);
        }
        __syncwarp();
        s_cand[warp][lane] = 0;
        __syncwarp();
        if (lane < total) s_cand[warp][place] = mine;
        __syncwarp();
        my_key = (uint32_t)(s_cand[warp][lane] >> 32);
        my_idx = ~(uint32_t)s_cand[warp][lane];
    } else {
        uint32_t taken = 0;                   // bit c·W + i: v[c][i] has been chosen
        for (int k = 0; k < K; ++k) {
            uint32_t best = 0, idx = FULL;
            for (int b = 0; b < C * W; ++b) { // from shared memory (this lane's own stores), so that no registers wait here
                const int at_b = b / W * CHUNK + lane * W + b % W;
                const uint32_t key = taken >> b & 1u ? 0u : score_key(s_row[warp][at_b]);
                if (key > best) {
                    best = key;
                    idx = (uint32_t)at_b;
                }
            }
            const uint32_t most = __reduce_max_sync(FULL, best);
            if (most <= KEY_MINUS_INF) break; // nothing above -inf is left
            const uint32_t first = __reduce_min_sync(FULL, best == most ? idx : FULL);
            if (idx == first) taken |= 1u << (idx / CHUNK * W + idx % W);
            if (lane == k) {
                my_key = most;
                my_idx = first;
            }
        }
    }

    const bool live = lane < K && my_key > KEY_MINUS_INF;
    const float mine = key_score(my_key);
    const float m = __shfl_sync(FULL, mine, 0);  // unused where lane 0 is not live
    const float ex = live ? expf(mine - m) : 0.0f;
    const float sum = warp_sum(ex);
    if (lane < K) {
        p[t * K + lane] = live ? ex / sum : 0.0f;
        ids[t * K + lane] = live ? (int32_t)my_idx : -1;
    }
}

// One warp per token: the row is zeroed with 16-byte stores, then the at most 32 places are written
// over it (ordered by __syncwarp; both meet in L2, so HBM sees each line once).
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(WARPS * 32)
    route_topk_bwd_kernel(const int32_t* __restrict__ ids, const float* __restrict__ p, const float* __restrict__ dp,
                          const int32_t* __restrict__ row_of, int64_t R, void* __restrict__ dlogits, int64_t T, int E,
                          int K) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * WARPS + warp;
    if (t >= T) return;
    int id = -1;
    float pk = 0.0f, dpk = 0.0f;
    if (lane < K) {
        id = ids[t * K + lane];
        int64_t at = t * K + lane;
        bool live = (uint32_t)id < (uint32_t)E;
        if (row_of) {
            at = row_of[at];
            live = live && at >= 0 && at < R;
        }
        if (live) {
            pk = p[t * K + lane];
            dpk = dp[at];
        } else {
            id = -1;
        }
    }
    if constexpr (VEC) {
        constexpr int W = BF16 ? 8 : 4;
        uint4* row = (uint4*)((char*)dlogits + t * E * (BF16 ? 2 : 4));
        for (int c = lane; c < E / W; c += 32) row[c] = make_uint4(0, 0, 0, 0);
    } else {
        for (int e = lane; e < E; e += 32) {
            if constexpr (BF16) ((uint16_t*)dlogits)[t * E + e] = 0;
            else ((float*)dlogits)[t * E + e] = 0.0f;
        }
    }
    const float dot = warp_sum(id >= 0 ? pk * dpk : 0.0f);
    __syncwarp();
    if (id >= 0) {
        const float d = pk * (dpk - dot);
        if constexpr (BF16) ((uint16_t*)dlogits)[t * E + id] = f32_to_bf16(d);
        else ((float*)dlogits)[t * E + id] = d;
    }
}

template <bool BF16, int W>
int launch_route(const void* logits, float* p, int32_t* ids, int64_t T, int E, int K, cudaStream_t stream) {
    const unsigned grid = (unsigned)((T + WARPS - 1) / WARPS);
    const int chunks = (E + 32 * W - 1) / (32 * W);
#define SITU_ROUTE_CASE(C)                                                                          \
    if (chunks <= C) {                                                                              \
        route_topk_kernel<BF16, W, C><<<grid, WARPS * 32, 0, stream>>>(logits, p, ids, T, E, K);    \
        const cudaError_t e = cudaGetLastError();                                                   \
        return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);                                       \
    }
    // few registers for few scores; 32·W·C covers E <= 1024 in every instance's largest C
    SITU_ROUTE_CASE(1)
    SITU_ROUTE_CASE(2)
    SITU_ROUTE_CASE(4)
    if constexpr (W <= 4) {
        SITU_ROUTE_CASE(7)
        SITU_ROUTE_CASE(8)
    }
    if constexpr (W == 1) {
        SITU_ROUTE_CASE(16)
        SITU_ROUTE_CASE(32)
    }
#undef SITU_ROUTE_CASE
    return SITU_GLU_INVALID_ARG;
}

int check_route(int type, int64_t T, int64_t E, int64_t K) {
    if (type != SITU_BF16 && type != SITU_FP32) return SITU_GLU_INVALID_ARG;
    if (T < 0 || T > INT32_MAX || E < 1 || E > SITU_MAX_EXPERTS || K < 1 || K > SITU_MAX_TOPK || K > E)
        return SITU_GLU_INVALID_ARG;
    return SITU_GLU_OK;
}

}  // namespace

extern "C" {

int situ_route_topk(const void* logits, int type, float* p, int32_t* ids, int64_t T, int64_t E, int64_t K,
                    cudaStream_t stream) {
    const int st = check_route(type, T, E, K);
    if (st != SITU_GLU_OK) return st;
    if (T == 0) return SITU_GLU_OK;
    const int64_t sz = type == SITU_BF16 ? 2 : 4;
    if (!logits || !p || !ids || !aligned(logits, (uintptr_t)sz) || !aligned(p, 4) || !aligned(ids, 4))
        return SITU_GLU_INVALID_ARG;
    const Range rl = range_of(logits, T * E * sz), rp = range_of(p, T * K * 4), ri = range_of(ids, T * K * 4);
    if (overlap(rp, rl) || overlap(ri, rl) || overlap(rp, ri)) return SITU_GLU_OVERLAP;
    const bool vec = aligned(logits, 16) && E * sz % 16 == 0;
    if (type == SITU_BF16)
        return vec ? launch_route<true, 8>(logits, p, ids, T, (int)E, (int)K, stream)
                   : launch_route<true, 1>(logits, p, ids, T, (int)E, (int)K, stream);
    return vec ? launch_route<false, 4>(logits, p, ids, T, (int)E, (int)K, stream)
               : launch_route<false, 1>(logits, p, ids, T, (int)E, (int)K, stream);
}

int situ_route_topk_bwd(const int32_t* ids, const float* p, const float* dp, const int32_t* row_of, int64_t R,
                        void* dlogits, int type, int64_t T, int64_t E, int64_t K, cudaStream_t stream) {
    const int st = check_route(type, T, E, K);
    if (st != SITU_GLU_OK) return st;
    if (row_of && (R < 0 || R > INT32_MAX)) return SITU_GLU_INVALID_ARG;
    if (T == 0) return SITU_GLU_OK;
    const int64_t sz = type == SITU_BF16 ? 2 : 4;
    const int64_t ndp = row_of ? R : T * K;
    if (!ids || !p || (!dp && ndp > 0) || !dlogits || !aligned(ids, 4) || !aligned(p, 4) || !aligned(dp, 4) ||
        !aligned(row_of, 4) || !aligned(dlogits, (uintptr_t)sz))
        return SITU_GLU_INVALID_ARG;
    const Range rd = range_of(dlogits, T * E * sz);
    if (overlap(rd, range_of(ids, T * K * 4)) || overlap(rd, range_of(p, T * K * 4)) ||
        (dp && overlap(rd, range_of(dp, ndp * 4))) || (row_of && overlap(rd, range_of(row_of, T * K * 4))))
        return SITU_GLU_OVERLAP;
    const unsigned grid = (unsigned)((T + WARPS - 1) / WARPS);
    const bool vec = aligned(dlogits, 16) && E * sz % 16 == 0;
    auto kernel = type == SITU_BF16 ? (vec ? route_topk_bwd_kernel<true, true> : route_topk_bwd_kernel<true, false>)
                                    : (vec ? route_topk_bwd_kernel<false, true> : route_topk_bwd_kernel<false, false>);
    kernel<<<grid, WARPS * 32, 0, stream>>>(ids, p, dp, row_of, R, dlogits, T, (int)E, (int)K);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

}  // extern "C"
