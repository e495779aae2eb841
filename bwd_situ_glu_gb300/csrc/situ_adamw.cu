// situ_adamw.cu — one AdamW step over many tensors on the device, states in fp32 or in 8 bits (include/situ_adamw.h, which
// has the formulas).
//
// HBM-bound: with fp32 gradients and a bf16 working copy 30 bytes a parameter (16 of them the states'), with 8-bit states and
// bf16 gradients 16. One launch for all tensors: their pointers travel as a kernel parameter (up to 32 KB), so a step needs
// no table on the device and can be captured. A block takes CHUNK elements of one tensor and finds it by bisection; a lane 8
// consecutive elements, half a warp a block of 128, whose largest values it finds by shuffles.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/situ_adamw.h"
#include "situ_device.cuh"
#include "situ_fp8.cuh"
#include "situ_host.h"

namespace {

using namespace situ;
using namespace situ_host;
using namespace situ_fp8;

// Instructions bound the step with states in 8 bits (some 80 an element: its IEEE root and quotient, the two codes, the random
// bits), so what counts is how many warps an SM has to choose from and how often a block's setup is paid: 201M elements, bf16
// gradients and copies, in 128-thread blocks, 10 an SM, 8 passes, 519 us (0.93 of the copy rate; without paired products 534);
// 8 or 12 blocks 552 / 535; 256 threads and 4 passes 600, one pass 732. States in fp32 run at the copy rate either way.
// A tensor with a pointer off its vectors takes one element at a time, all its arrays alike: 245M elements whose gradients lie at odd places of
// one buffer 2180 us (8-bit states) and 3390 (fp32) instead of 639 and 1043. Zeros everywhere, states and gradients, take 891 instead of 639
// in 8 bits.
constexpr int TPB = 128, BLOCKS_PER_SM = 10;
constexpr int STEP = TPB * 8;                // elements of one pass of a block
constexpr int PASSES = 8;
constexpr int CHUNK = STEP * PASSES;         // elements of a block: a multiple of 128

struct Entry {
    float* w;
    const void* g;
    void *m, *v;
    uint8_t *ms, *vs;
    uint16_t* work;
    int64_t n;                               // its sign: negative where the pointers are off the vectors
};

template <int CAP>
struct Table {
    Entry e[CAP];
    int first[CAP];                          // first block of each tensor
    int count;
};
constexpr int MAX_TENSORS = 448;
static_assert(sizeof(Table<MAX_TENSORS>) + 64 <= 32764, "kernel parameters");

using Coefs = situ_adamw_coefficients;

__host__ __device__ inline uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x9E3779B1u;                        // the fractions of the golden ratio and of sqrt 2
    x ^= x >> 15;
    x *= 0x6A09E667u;
    return x ^ (x >> 16);
}

// The E4M3 code of a = |y|·2^-120, |y| <= 448, rounded at random, in the bits from 20 on: fp32 with its exponent moved to
// E4M3's has the code above its lowest 20 bits, for subnormal codes as for normal ones. To those 16 random bits are added, and
// four zeros.
__device__ __forceinline__ uint32_t random_code(float a, uint32_t bits16) { return bits16 * 16u + __float_as_uint(a); }

// The upper bytes of four words.
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// One moment's 8 values to codes: q (code in the upper byte), returns the block's scale byte. SHIFT: which 16 of the
// random bits. LIFT: the values are at least 0, and what is above 0 gets a code above 0. All lanes of the warp.
template <int SHIFT, bool LIFT>
__device__ __forceinline__ int encode_moment(const float (&x)[8], const uint32_t (&r)[8], uint32_t (&q)[8]) {
    uint32_t top = 0;                        // largest |x| by its bits: infinities and NaN are above all numbers
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, LIFT ? __float_as_uint(x[k]) : __float_as_uint(x[k]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const auto bits16 = [&](int k) { return SHIFT ? r[k] >> 16 : r[k] & 0xFFFFu; };
    // 2^11 and less: |x|·2^(127-b)·2^-120 is one multiplication by a number
    if (__all_sync(0xffffffffu, top < 0x45000000u)) {
        const int b = scale_byte(__uint_as_float(top));
        const float f = __uint_as_float((uint32_t)(134 - b) << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            q[k] = random_code(__fmul_rn(fabsf(x[k]), f), bits16(k));
            if (LIFT) q[k] = max(q[k], x[k] > 0.0f ? 1u << 20 : 0u);
            q[k] <<= 4;
            if (!LIFT) q[k] |= __float_as_uint(__fadd_rn(x[k], 0.0f)) & 0x80000000u;     // no sign on -0
        }
        return b;
    }
    float amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, finite_abs(x[k]));
    const int b = scale_byte(halfwarp_max(amax));
    const float inv = inverse_scale(b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float y = __fmul_rn(x[k], inv), a = fabsf(y);
        uint32_t c = random_code(__fmul_rn(a, 0x1p-120f), bits16(k));
        if (LIFT && y > 0.0f) c = max(c, 1u << 20);
        if (!(a < __int_as_float(0x7F800000))) c = 0x07F00000u;
        q[k] = (c << 4) | (y < 0.0f ? 0x80000000u : 0u);
    }
    return b;
}

__device__ __forceinline__ float2 two(const float (&x)[8], int k) { return make_float2(x[k], x[k + 1]); }
// Products by the paired instruction, each half rounded as the single one; sums one by one: ptxas makes one operation of a paired
// product and a paired sum, whatever rounding they ask for.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }
__device__ __forceinline__ void put(float (&x)[8], int k, float2 f) {
    x[k] = f.x;
    x[k + 1] = f.y;
}

template <bool BF16_GRAD, bool EIGHT, int CAP>
__global__ void __launch_bounds__(TPB, BLOCKS_PER_SM)
    adamw_kernel(const __grid_constant__ Table<CAP> table, const Coefs given, const Coefs* __restrict__ from_device,
                 const float* __restrict__ grad_scale) {
    int lo = 0, hi = table.count - 1;        // last tensor whose first block is <= this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table.first[mid] <= (int)blockIdx.x) lo = mid; else hi = mid - 1;
    }
    const Entry& t = table.e[lo];
    const bool vectors = t.n >= 0;
    const int64_t n = vectors ? t.n : -t.n;
    const Coefs c = from_device ? *from_device : given;
    const float gs = grad_scale ? *grad_scale : 1.0f;
    const int64_t begin = (int64_t)((int)blockIdx.x - table.first[lo]) * CHUNK;
#pragma unroll 1
    for (int p = 0; p < PASSES; ++p) {
        const int64_t i0 = begin + p * STEP + (int64_t)threadIdx.x * 8;
        if (begin + p * STEP >= n) break;    // the same for the block
        const bool full = vectors && i0 + 8 <= n;
        const int live = i0 >= n ? 0 : (int)min((int64_t)8, n - i0);
        float w[8], g[8], m[8], v[8];
        if (full) {
            const Vec<8> wv = ld_stream<8, false>((const Vec<8>*)(t.w + i0));
            if constexpr (BF16_GRAD) {
                const Vec<4> gv = ld_stream<4, true>((const Vec<4>*)((const uint16_t*)t.g + i0));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    g[2 * k] = bf16_lo(gv.w[k]);
                    g[2 * k + 1] = bf16_hi(gv.w[k]);
                }
            } else {
                const Vec<8> gv = ld_stream<8, true>((const Vec<8>*)((const float*)t.g + i0));
#pragma unroll
                for (int k = 0; k < 8; ++k) g[k] = __uint_as_float(gv.w[k]);
            }
            if constexpr (EIGHT) {
                decode8(*(const uint2*)((const uint8_t*)t.m + i0), m);
                decode8(*(const uint2*)((const uint8_t*)t.v + i0), v);
            } else {
                const Vec<8> mv = ld_stream<8, false>((const Vec<8>*)((const float*)t.m + i0));
                const Vec<8> vv = ld_stream<8, false>((const Vec<8>*)((const float*)t.v + i0));
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    m[k] = __uint_as_float(mv.w[k]);
                    v[k] = __uint_as_float(vv.w[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = __uint_as_float(wv.w[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                w[k] = g[k] = m[k] = v[k] = 0.0f;
                if (k < live) {
                    w[k] = t.w[i0 + k];
                    g[k] = BF16_GRAD ? bf16_to_f32(((const uint16_t*)t.g)[i0 + k]) : ((const float*)t.g)[i0 + k];
                    if constexpr (EIGHT) {
                        float none;
                        e4m3x2_to_f32(((const uint8_t*)t.m)[i0 + k], m[k], none);
                        e4m3x2_to_f32(((const uint8_t*)t.v)[i0 + k], v[k], none);
                    } else {
                        m[k] = ((const float*)t.m)[i0 + k];
                        v[k] = ((const float*)t.v)[i0 + k];
                    }
                }
            }
        }
        if constexpr (EIGHT) {
            const float sm = live ? scale_value(t.ms[i0 / QBLOCK]) : 1.0f, sv = live ? scale_value(t.vs[i0 / QBLOCK]) : 1.0f;
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                put(m, k, mul2(two(m, k), both(sm)));
                const float2 root = mul2(two(v, k), both(sv));
                put(v, k, mul2(root, root));
            }
        }
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            float2 gk = two(g, k);
            if (grad_scale) gk = mul2(gk, both(gs));
            const float2 m1 = add2(mul2(both(c.b1), two(m, k)), mul2(both(c.c1), gk));
            const float2 v1 = add2(mul2(both(c.b2), two(v, k)), mul2(both(c.c2), mul2(gk, gk)));
            const float2 root = make_float2(__fsqrt_rn(v1.x), __fsqrt_rn(v1.y));
            const float2 q = add2(mul2(root, both(c.r)), both(c.eps));
            const float2 ratio = make_float2(__fdiv_rn(m1.x, q.x), __fdiv_rn(m1.y, q.y));
            // w1 - s·ratio as w1 + (-s)·ratio: the same product but for its sign
            put(w, k, add2(mul2(two(w, k), both(c.d)), mul2(both(-c.s), ratio)));
            put(m, k, m1);
            put(v, k, EIGHT ? root : v1);
        }
        if constexpr (EIGHT) {               // lanes without elements hold zeros and take part
            uint32_t r[8], qm[8], qv[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = mix((uint32_t)i0 + (uint32_t)k + c.key);
            const int bm = encode_moment<0, false>(m, r, qm), bv = encode_moment<16, true>(v, r, qv);
            if (full) {
                *(uint2*)((uint8_t*)t.m + i0) = make_uint2(codes4(qm[0], qm[1], qm[2], qm[3]), codes4(qm[4], qm[5], qm[6], qm[7]));
                *(uint2*)((uint8_t*)t.v + i0) = make_uint2(codes4(qv[0], qv[1], qv[2], qv[3]), codes4(qv[4], qv[5], qv[6], qv[7]));
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < live) {
                        ((uint8_t*)t.m)[i0 + k] = (uint8_t)(qm[k] >> 24);
                        ((uint8_t*)t.v)[i0 + k] = (uint8_t)(qv[k] >> 24);
                    }
            }
            if (live && i0 % QBLOCK == 0) {
                t.ms[i0 / QBLOCK] = (uint8_t)bm;
                t.vs[i0 / QBLOCK] = (uint8_t)bv;
            }
        }
        if (full) {
            Vec<8> o;
#pragma unroll
            for (int k = 0; k < 8; ++k) o.w[k] = __float_as_uint(w[k]);
            st_stream<8>((Vec<8>*)(t.w + i0), o);
            if (t.work) {
                Vec<4> b;
#pragma unroll
                for (int k = 0; k < 4; ++k) b.w[k] = pack_bf16x2(w[2 * k], w[2 * k + 1]);
                st_stream<4>((Vec<4>*)(t.work + i0), b);
            }
            if constexpr (!EIGHT) {
#pragma unroll
                for (int k = 0; k < 8; ++k) o.w[k] = __float_as_uint(m[k]);
                st_stream<8>((Vec<8>*)((float*)t.m + i0), o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o.w[k] = __float_as_uint(v[k]);
                st_stream<8>((Vec<8>*)((float*)t.v + i0), o);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < live) {
                    t.w[i0 + k] = w[k];
                    if (t.work) t.work[i0 + k] = f32_to_bf16(w[k]);
                    if constexpr (!EIGHT) {
                        ((float*)t.m)[i0 + k] = m[k];
                        ((float*)t.v)[i0 + k] = v[k];
                    }
                }
        }
    }
}

// ---------------------------------------------------------------- host side

bool params_ok(const situ_adam_params* hp) {
    if (!hp) return false;
    const double lr = hp->lr, b1 = hp->beta1, b2 = hp->beta2, eps = hp->eps, wd = hp->weight_decay;
    return isfinite(lr) && lr >= 0.0 && isfinite(b1) && b1 >= 0.0 && b1 < 1.0 && isfinite(b2) && b2 >= 0.0 && b2 < 1.0 &&
           isfinite(eps) && eps > 0.0 && isfinite(wd) && wd >= 0.0 && hp->step >= 1;
}

Coefs coefficients_of(const situ_adam_params& hp, uint32_t seed) {
    Coefs k;
    k.b1 = (float)hp.beta1;
    k.b2 = (float)hp.beta2;
    k.eps = (float)hp.eps;
    k.c1 = (float)(1.0 - hp.beta1);
    k.c2 = (float)(1.0 - hp.beta2);
    k.s = (float)(hp.lr / (1.0 - pow(hp.beta1, (double)hp.step)));
    k.r = (float)(1.0 / sqrt(1.0 - pow(hp.beta2, (double)hp.step)));
    k.d = (float)(1.0 - hp.lr * hp.weight_decay);         // 1 without decay: w·1 is w
    k.key = mix(seed * 0x9E3779B1u);
    return k;
}

struct Span {
    uintptr_t lo, hi;
    bool written;
};

// Everything that situ_adamw_step says of its tensors; the vectors' alignment into off_vectors.
int check_tensors(const situ_adamw_tensor* t, int64_t count, int grad_type, int state_type, const float* grad_scale,
                  const Coefs* coefficients, std::vector<char>& off_vectors) {
    const int64_t gsz = grad_type == SITU_BF16 ? 2 : 4;
    const bool eight = state_type == SITU_E4M3;
    std::vector<Span> spans;
    spans.reserve((size_t)count * 7 + 2);
    off_vectors.assign((size_t)count, 0);
    const auto add = [&](const void* p, int64_t bytes, bool written) {
        spans.push_back(Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, written});
    };
    for (int64_t i = 0; i < count; ++i) {
        const situ_adamw_tensor& x = t[i];
        if (x.n < 0 || x.n >= (int64_t)1 << 42) return SITU_GLU_INVALID_ARG;
        if (x.n == 0) continue;
        if (!x.w || !x.grad || !x.m || !x.v || (eight && (!x.m_scales || !x.v_scales))) return SITU_GLU_INVALID_ARG;
        if (!aligned(x.w, 4) || !aligned(x.grad, (uintptr_t)gsz) || !aligned(x.work, 2) ||
            (!eight && (!aligned(x.m, 4) || !aligned(x.v, 4))))
            return SITU_GLU_INVALID_ARG;
        off_vectors[(size_t)i] = !aligned(x.w, 32) || !aligned(x.grad, grad_type == SITU_BF16 ? 16 : 32) || !aligned(x.work, 16) ||
                                 !aligned(x.m, eight ? 8 : 32) || !aligned(x.v, eight ? 8 : 32);
        add(x.w, x.n * 4, true);
        add(x.grad, x.n * gsz, false);
        add(x.m, x.n * (eight ? 1 : 4), true);
        add(x.v, x.n * (eight ? 1 : 4), true);
        if (eight) {
            add(x.m_scales, (x.n + QBLOCK - 1) / QBLOCK, true);
            add(x.v_scales, (x.n + QBLOCK - 1) / QBLOCK, true);
        }
        if (x.work) add(x.work, x.n * 2, true);
    }
    if (grad_scale) add(grad_scale, 4, false);
    if (coefficients) add(coefficients, sizeof(Coefs), false);
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t written = 0, read = 0;         // the furthest ends so far
    for (const Span& s : spans) {
        if (s.lo < written || (s.written && s.lo < read)) return SITU_GLU_OVERLAP;
        (s.written ? written : read) = std::max(s.written ? written : read, s.hi);
    }
    return SITU_GLU_OK;
}

template <bool BF16_GRAD, bool EIGHT, int CAP>
int launch_some(const situ_adamw_tensor* const* t, const char* off, int count, int blocks, const Coefs& given, const Coefs* from_device,
                const float* grad_scale, cudaStream_t stream) {
    Table<CAP> table;
    table.count = count;
    int first = 0;
    for (int i = 0; i < count; ++i) {
        const situ_adamw_tensor& x = *t[i];
        table.e[i] = Entry{x.w, x.grad, x.m, x.v, x.m_scales, x.v_scales, (uint16_t*)x.work, off[i] ? -x.n : x.n};
        table.first[i] = first;
        first += (int)((x.n + CHUNK - 1) / CHUNK);
    }
    adamw_kernel<BF16_GRAD, EIGHT, CAP><<<blocks, TPB, 0, stream>>>(table, given, from_device, grad_scale);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SITU_GLU_OK : cuda_fail(e);
}

template <bool BF16_GRAD, bool EIGHT>
int launch_all(const situ_adamw_tensor* tensors, int64_t count, const std::vector<char>& off_vectors, const Coefs& given,
               const Coefs* from_device, const float* grad_scale, cudaStream_t stream) {
    const situ_adamw_tensor* t[MAX_TENSORS];
    char off[MAX_TENSORS];
    int some = 0;
    int64_t blocks = 0;
    const auto flush = [&]() -> int {
        if (some == 0) return SITU_GLU_OK;
        const auto go = [&](auto launch) { return launch(t, off, some, (int)blocks, given, from_device, grad_scale, stream); };
        // the parameter is copied for each launch: as small as the tensors need
        const int st = some <= 16   ? go(launch_some<BF16_GRAD, EIGHT, 16>)
                       : some <= 96 ? go(launch_some<BF16_GRAD, EIGHT, 96>)
                                    : go(launch_some<BF16_GRAD, EIGHT, MAX_TENSORS>);
        some = 0;
        blocks = 0;
        return st;
    };
    for (int64_t i = 0; i < count; ++i) {
        if (tensors[i].n == 0) continue;
        const int64_t more = (tensors[i].n + CHUNK - 1) / CHUNK;        // below 2^29
        if (some == MAX_TENSORS || blocks + more > INT32_MAX) {
            const int st = flush();
            if (st != SITU_GLU_OK) return st;
        }
        t[some] = &tensors[i];
        off[some++] = off_vectors[(size_t)i];
        blocks += more;
    }
    return flush();
}

}  // namespace

extern "C" {

int situ_adamw_coefficients_of(const situ_adam_params* hp, uint32_t seed, situ_adamw_coefficients* out) {
    if (!params_ok(hp) || !out) return SITU_GLU_INVALID_ARG;
    *out = coefficients_of(*hp, seed);
    return SITU_GLU_OK;
}

int situ_adamw_step(const situ_adamw_tensor* tensors, int64_t count, int grad_type, int state_type, const situ_adam_params* hp,
                    uint32_t seed, const situ_adamw_coefficients* coefficients, const float* grad_scale, cudaStream_t stream) {
    if (count < 0 || count > INT32_MAX || (count && !tensors) || (grad_type != SITU_BF16 && grad_type != SITU_FP32) ||
        (state_type != SITU_FP32 && state_type != SITU_E4M3) || !aligned(coefficients, 4) || !aligned(grad_scale, 4))
        return SITU_GLU_INVALID_ARG;
    if (!coefficients && !params_ok(hp)) return SITU_GLU_INVALID_ARG;
    try {
        std::vector<char> off_vectors;
        const int st = check_tensors(tensors, count, grad_type, state_type, grad_scale, coefficients, off_vectors);
        if (st != SITU_GLU_OK) return st;
        const Coefs given = coefficients ? Coefs{} : coefficients_of(*hp, seed);
        const auto go = [&](auto launch) { return launch(tensors, count, off_vectors, given, coefficients, grad_scale, stream); };
        if (grad_type == SITU_BF16)
            return state_type == SITU_E4M3 ? go(launch_all<true, true>) : go(launch_all<true, false>);
        return state_type == SITU_E4M3 ? go(launch_all<false, true>) : go(launch_all<false, false>);
    } catch (const std::bad_alloc&) {        // the host's lists: nothing has been launched
        return cuda_fail(cudaErrorMemoryAllocation);
    }
}

}  // extern "C"
