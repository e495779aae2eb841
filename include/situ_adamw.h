/* situ_adamw.h — one AdamW step over many tensors in device memory, with states in fp32 or in 8 bits, in the same C
 * ABI as situ_glu.h (libsitu_glu.so). (situ_adam_stream_step is the step for state in host memory.)
 *
 * One step per element, as single IEEE fp32 operations in the order of situ_adam_update_host (constants formed in double
 * from the hyper-parameters and rounded to fp32 once: b1, b2, eps, c1 = 1 - beta1, c2 = 1 - beta2,
 * s = lr / (1 - beta1^step), r = 1 / sqrt(1 - beta2^step), d = 1 - lr·weight_decay):
 *   g  = grad, or grad·grad_scale where that is given
 *   w1 = weight_decay > 0 ? w·d : w
 *   m1 = b1·m + c1·g;   v1 = b2·v + c2·(g·g);   q = sqrt(v1)·r + eps;   w2 = w1 - s·(m1/q)
 *   stored: w = w2, work (if any) = bf16(w2) to nearest even, and the states.
 *
 * States in fp32 (SITU_FP32): m = m1, v = v1.
 * States in 8 bits (SITU_E4M3): m, and the root of v, as E4M3 codes with a scale byte for each 128 consecutive elements of
 * a tensor, as situ_quant_fp8 chooses it (situ_fp8.h), so v = (code·2^(b-127))². Of the two codes around a value the step takes
 * the upper one (in magnitude) with the probability of the value's place between them, in 2^-16: a moment that moves by
 * less than a code's step (v by 1 - beta2 of itself) still moves, on average by what it should. Rounded to nearest it would stay
 * where it is. A root above 0 gets a code above 0 (m/0 would throw its weight off); a value that is not finite gets 0x7F (NaN).
 * What that makes of v. The mean kept is the root's, so v itself comes out high. Where the root's code is one of E4M3's normal numbers
 * (2^-6·2^(b-127) or more), v gains up to (1 - beta2)/16·|g² - v| a step on average. In the long run its mean lies above that of states in
 * fp32 by 0.4 % for a constant gradient, by 2.5 to 4.6 % for independent normal ones (beta2 0.95 to 0.999), by 3.5 to 7.2 % for normal ones
 * in one step of ten and 0 between, and never by more than 2/15; one element's v scatters by 0.24 to 0.43 of it. Below, at codes k = 1 .. 7,
 * the gain is up to (1 - beta2)/(2k)·|g² - v|, and code 1 is a floor: the root of an element that ever had a gradient stays at
 * 2^-9·2^(b-127) or above, 2^-17.8 to 2^-16.8 of its block's largest, so that elements so small step less than with states in fp32.
 * The 16 bits are those of mix(i + key) for element i of its tensor (modulo 2^32): the lower half for m, the upper for
 * v; key = mix(seed·0x9E3779B1), and mix(x) is x ^= x>>16, x *= 0x9E3779B1, x ^= x>>15, x *= 0x6A09E667, x ^= x>>16. No result
 * depends on timing, on the order of the tensors or on how they are split over calls.
 */
#ifndef SITU_ADAMW_H
#define SITU_ADAMW_H

#include "situ_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SITU_E4M3 = 2 };

/* One tensor: n >= 0 elements, all pointers on the device. */
typedef struct {
    float* w;            /* updated */
    const void* grad;    /* of grad_type */
    void* m;             /* fp32 or codes, updated */
    void* v;
    uint8_t* m_scales;   /* [ceil(n/128)] with states in 8 bits (else NULL), updated */
    uint8_t* v_scales;
    void* work;          /* bf16 working copy, written; or NULL */
    int64_t n;
} situ_adamw_tensor;

/* What a step computes with, as it is read from the device: for a step captured in a graph, whose hyper-parameters, step
 * count and seed change from replay to replay. */
typedef struct {
    float b1, b2, eps, c1, c2, s, r, d;
    uint32_t key;
} situ_adamw_coefficients;
int situ_adamw_coefficients_of(const situ_adam_params* hp, uint32_t seed, situ_adamw_coefficients* out);

/* The step over tensors[0 .. count-1] (a host array, read before the call returns). grad_type SITU_BF16 or SITU_FP32,
 * state_type SITU_FP32 or SITU_E4M3, the same for all. hp and seed, or, with coefficients (device, 4-byte aligned) given, what
 * they say (hp may then be NULL). grad_scale: one fp32 on the device, or NULL. Any alignment of the element types (vectors where
 * a tensor's pointers are on 32 bytes, those of bf16 on 16 and of codes on 8). No two tensors share memory that the step writes, and no
 * gradient shares memory with it (SITU_GLU_OVERLAP). Kernel launches: one for each 448 tensors. */
int situ_adamw_step(const situ_adamw_tensor* tensors, int64_t count, int grad_type, int state_type, const situ_adam_params* hp,
                    uint32_t seed, const situ_adamw_coefficients* coefficients, const float* grad_scale, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SITU_ADAMW_H */
