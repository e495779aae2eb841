// situ_linear.cuh — what the linear operator's forward and gradient kernels share: the activations and
// their derivatives, and the prefix over experts.
#pragma once

#include <math.h>
#include <stdint.h>

#include "../../include/situ_moe.h"
#include "situ_host.h"

namespace situ_linear {

constexpr uint32_t FULL_MASK = 0xffffffffu;

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The normal distribution's Φ(z) and e^{-z²/2}. For z <= 0, Φ(z)·e^{z²/2} is smooth and falls like 1/|z|: t·P(t) with
// t = 1/(1 + p|z|), P of degree 6 and p chosen for the least maximal RELATIVE error over 0 <= |z| <= 14.5, where e^{-z²/2}
// leaves fp32 (a linear programme over the coefficients against erfc in 64 bits: 8e-7). So Φ on the left side, and
// gelu with it, has a small relative error too: 8e-7 and the rounding of z²/2 in the exponential, together below
// 3e-6 + z²·1.2e-7. One ex2, one rcp and some ten multiply-adds; two
// terms fewer would leave 3e-5. (4099 x 3584 x 1000 with gelu: 36.3 us; with five terms of small absolute error 35.6.)
constexpr float PHI_P = 0.363f;
__device__ __forceinline__ constexpr float phi_c(int i) {
    constexpr float c[7] = {0.144895628f, 0.143201366f, 0.13898167f, 0.0308226421f, 0.173150882f, -0.17913875f, 0.0480869599f};
    return c[i];
}
struct Normal {
    float cdf, e;
};
__device__ __forceinline__ Normal normal(float z) {
    const float e = ex2_approx(z * z * -0.72134752044448170f);   // e^{-z²/2}
    const float t = rcp_approx(fmaf(fabsf(z), PHI_P, 1.0f));
    float q = fmaf(t, phi_c(6), phi_c(5));
#pragma unroll
    for (int i = 4; i >= 0; --i) q = fmaf(q, t, phi_c(i));
    q = q * t * e;                           // Φ(-|z|)
    return Normal{z >= 0.0f ? 1.0f - q : q, e};
}

// act(z) in fp32. silu: z·σ(z), with an exponential that overflows to +inf (z/inf = -0) below z ≈ -88.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == SITU_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == SITU_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    if constexpr (ACT == SITU_ACT_GELU) return z * normal(z).cdf;
    return z;
}

// act of two values with the paired fp32 instructions (one issue slot for the same operation on both; each half
// rounds as the scalar one): some ten instead of sixteen slots a value for gelu, whose epilogue otherwise takes as long
// as the products at K = 1000.
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }
template <int ACT>
__device__ __forceinline__ float2 act_pair(float2 z) {
    if constexpr (ACT == SITU_ACT_RELU) return make_float2(act_value<ACT>(z.x), act_value<ACT>(z.y));
    if constexpr (ACT == SITU_ACT_SILU) {
        const float2 a = __fmul2_rn(z, both(-1.4426950408889634f));
        const float2 d = __fadd2_rn(make_float2(ex2_approx(a.x), ex2_approx(a.y)), both(1.0f));
        return __fmul2_rn(z, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    }
    if constexpr (ACT == SITU_ACT_GELU) {    // as normal()
        const float2 x = __fmul2_rn(__fmul2_rn(z, z), both(-0.72134752044448170f));
        const float2 d = __ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), both(PHI_P), both(1.0f));
        const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        float2 q = __ffma2_rn(t, both(phi_c(6)), both(phi_c(5)));
#pragma unroll
        for (int i = 4; i >= 0; --i) q = __ffma2_rn(q, t, both(phi_c(i)));
        q = __fmul2_rn(__fmul2_rn(q, t), make_float2(ex2_approx(x.x), ex2_approx(x.y)));
        const float2 p = __ffma2_rn(q, both(-1.0f), both(1.0f));
        return __fmul2_rn(z, make_float2(z.x >= 0.0f ? p.x : q.x, z.y >= 0.0f ? p.y : q.y));
    }
    return z;
}

// act'(z) in fp32.
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == SITU_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if constexpr (ACT == SITU_ACT_SILU) {    // σ + z·σ·(1 − σ)
        const float s = rcp_approx(1.0f + ex2_approx(z * -1.4426950408889634f));
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == SITU_ACT_GELU) {    // Φ(z) + z·φ(z)
        const Normal n = normal(z);
        return fmaf(z * 0.39894228040143268f, n.e, n.cdf);
    }
    return 1.0f;
}

// start[1 .. E] holds counts: their inclusive prefix in place, by one warp (each lane a segment).
__device__ __forceinline__ void prefix_in_place(int* start, int E, int lane) {
    const int seg = (E + 31) / 32;
    const int b = 1 + lane * seg, en = min(E + 1, b + seg);
    int sum = 0;
    for (int i = b; i < en; ++i) sum += start[i];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL_MASK, incl, o);
        if (lane >= o) incl += v;
    }
    int run = incl - sum;
    for (int i = b; i < en; ++i) {
        run += start[i];
        start[i] = run;
    }
}

// ---------------------------------------------------------------- host side

inline int sm_count(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    return e == cudaSuccess ? SITU_GLU_OK : situ_host::cuda_fail(e);
}

// Sizes shared by the product and its gradients. Row numbers are 32-bit, those past the last row that a chunk rounded up
// (32 rows) or the end of a split contraction (at most 16 blocks of 64) reaches among them.
constexpr int64_t MAX_ROWS = INT32_MAX - 1024;
inline int check_linear(int64_t E, const void* offsets, int64_t R, int64_t N, int64_t K) {
    if (R < 0 || R > MAX_ROWS || N < 8 || N % 8 != 0 || K < 8 || K % 8 != 0 || E < 1 || E > SITU_MAX_EXPERTS)
        return SITU_GLU_INVALID_ARG;
    if (N > INT32_MAX / 4 || K > INT32_MAX / 4 || E * N > INT32_MAX || E * K > INT32_MAX) return SITU_GLU_INVALID_ARG;
    if (!offsets && E != 1) return SITU_GLU_INVALID_ARG;
    return SITU_GLU_OK;
}

}  // namespace situ_linear
