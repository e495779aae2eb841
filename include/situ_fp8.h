/* situ_fp8.h — products in 8 bits for the expert layer, in the same C ABI as situ_moe.h
 * (libsitu_glu.so): block-scaled quantisation, and the per-expert (or dense) matrix product of
 * quantised rows and weights with its input gradient.
 *
 * The format. A value is an E4M3 code (OCP: 1 sign, 4 exponent, 3 mantissa bits; 0x7F is NaN, no
 * infinity) times the scale of its block of 128 consecutive elements of a row, or of 128 x 128 of a
 * weight. A scale is a byte b that stands for 2^(b - 127) (E8M0; 255 is NaN). Powers of two are what the
 * block-scaled tensor-core instruction takes as they are, and nothing is rounded but the code.
 * (situ_glu_fwd_save_fp8 keeps fp32 scales: its codes are never an operand.)
 *
 * Conventions are those of situ_moe.h: device pointers, contiguous row-major tensors, the caller owns
 * every buffer, work is enqueued on `stream` without a host wait, every argument is checked on the
 * host before any launch, and the result is a status code.
 */
#ifndef SITU_FP8_H
#define SITU_FP8_H

#include "situ_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- quantisation -------------------------------------------------------------------------
 * x [E, R, D] of `type` (SITU_BF16 or SITU_FP32) -> codes uint8 [E, R, D] and scales uint8
 * [E, ceil(R / block_rows), ceil(D / 128)], block_rows 1 (the rows of a product) or 128 (a weight).
 * Over a block's finite values, b is the least byte >= 1 with max |x| <= 448·2^(b-127) (1 where
 * there is no other value than 0), and the code is x·2^(127-b) rounded to nearest, ties to even; a value that is not
 * finite gets the code 0x7F. Fully determined: no step but the code rounds. E, R >= 0, D >= 1,
 * E·R·D < 2^62. Any alignment of the element type (16-byte vectors where D and the pointers allow). */
int situ_quant_fp8(const void* x, int type, uint8_t* codes, uint8_t* scales, int64_t E, int64_t R, int64_t D,
                   int block_rows, cudaStream_t stream);

/* x = code·2^(b-127), rounded to `type` to nearest even (exact in fp32; in bf16 where it is at least 2^-126 or has
 * its bits above 2^-133). The codes 0x7F and 0xFF, and a block whose byte is 255, give NaN. */
int situ_dequant_fp8(const uint8_t* codes, const uint8_t* scales, void* x, int type, int64_t E, int64_t R, int64_t D,
                     int block_rows, cudaStream_t stream);

/* ---- matrix product of quantised rows and weights ------------------------------------------
 * As situ_linear_fwd, with a [R, K] and w [E, N, K] (the nn.Linear layout) as codes and scales of
 * situ_quant_fp8 with block_rows 1 and 128: a_scales [R, ceil(K/128)], w_scales [E, ceil(N/128),
 * ceil(K/128)]. The products of codes and their scaling are exact, the sum over K is kept in fp32. bias, residual, act, out, pre,
 * expert_offsets and status are those of situ_linear_fwd. N % 16 == 0, K % 16 == 0; 1 <= E <= 1024;
 * R <= 2^31 - 1025; a, w, residual, out and pre 16-byte aligned. A NaN code or scale gives NaN in the row
 * (of a) or the output columns (of w) that use it, nowhere else. */
int situ_linear_fp8_fwd(const uint8_t* a, const uint8_t* a_scales, const uint8_t* w, const uint8_t* w_scales,
                        const int64_t* expert_offsets, int64_t E, const float* bias, const void* residual, int act, void* out,
                        int out_type, void* pre, int* status, int64_t R, int64_t N, int64_t K, cudaStream_t stream);

/* da bf16 [R, K] = dz·W_e (fp32 accumulation, rounded once) for dz [R, N] as codes and scales with block_rows 1
 * (dz_scales [R, ceil(N/128)]); the weights' codes and scales are the forward's. The other arguments as
 * situ_linear_fp8_fwd. (The weight gradient is situ_linear_wgrad of the unquantised dz and the decoded rows,
 * which bf16 holds exactly.) */
int situ_linear_fp8_dgrad(const uint8_t* dz, const uint8_t* dz_scales, const uint8_t* w, const uint8_t* w_scales,
                          const int64_t* expert_offsets, int64_t E, void* da, int* status, int64_t R, int64_t N, int64_t K,
                          cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SITU_FP8_H */
