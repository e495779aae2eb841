// situ_fp8.cuh — the 8-bit block format on the device: E4M3 codes with a power-of-two scale (a byte b for 2^(b-127)) for
// each 128 elements (include/situ_fp8.h). Shared by the quantiser, the products and the optimizer's states.
#pragma once

#include <stdint.h>

#include "situ_device.cuh"

namespace situ_fp8 {

constexpr int QBLOCK = 128;                  // elements of a row (or rows and columns of a weight) that share a scale

// |x|, or 0 for what is not finite.
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < __int_as_float(0x7F800000) ? a : 0.0f;
}

// Least b >= 1 with amax <= 448·2^(b-127), for finite amax >= 0: 448 = 1.75·2^8, so b is amax's exponent less 8, one
// more where its mantissa is above that of 1.75. At most 247; 1 keeps 2^(b-127) and 2^(127-b) normal.
__device__ __forceinline__ int scale_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int b = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b > 1 ? b : 1;
}

__device__ __forceinline__ float inverse_scale(int b) { return __uint_as_float((uint32_t)(254 - b) << 23); }   // b 1 .. 253

// Any byte: 0 is 2^-127, 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
    const uint32_t u = b == 0 ? 0x00400000u : b == 255 ? 0x7FFFFFFFu : b << 23;
    return __uint_as_float(u);
}

// Codes of two values (low byte lo): nearest, ties to even; not finite -> 0x7F.
__device__ __forceinline__ uint32_t encode2(float lo, float hi, float inv) {
    const float nan = __int_as_float(0x7FFFFFFF), inf = __int_as_float(0x7F800000);
    lo = fabsf(lo) < inf ? lo * inv : nan;
    hi = fabsf(hi) < inf ? hi * inv : nan;
    return situ::e4m3x2_from_f32(lo, hi);
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
    return make_uint2(encode2(f[0], f[1], inv) | (encode2(f[2], f[3], inv) << 16),
                      encode2(f[4], f[5], inv) | (encode2(f[6], f[7], inv) << 16));
}

__device__ __forceinline__ void decode8(uint2 q, float (&f)[8]) {
    situ::e4m3x2_to_f32((uint16_t)(q.x & 0xFFFFu), f[0], f[1]);
    situ::e4m3x2_to_f32((uint16_t)(q.x >> 16), f[2], f[3]);
    situ::e4m3x2_to_f32((uint16_t)(q.y & 0xFFFFu), f[4], f[5]);
    situ::e4m3x2_to_f32((uint16_t)(q.y >> 16), f[6], f[7]);
}

}  // namespace situ_fp8
