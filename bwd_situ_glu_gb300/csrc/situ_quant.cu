// situ_quant.cu — block-scaled quantisation to E4M3 with power-of-two scales, and back (include/situ_fp8.h).
//
// A block's scale is the least power of two that brings its largest finite value to 448 or below. 448 is
// 1.75·2^8, so its exponent follows from the bits of that value alone, and x·2^-e is exact: the code's rounding
// (cvt.rn.satfinite.e4m3x2) is the only one. One read of x, one write of codes; HBM-bound: 65537 x 3584 bf16 rows 112 us (0.94
// of the copy rate), from fp32 190 us (0.93), weights of 56 x 3584 x 2048 from fp32 335 us (0.92), from bf16 273 us (0.68), 16384 x 2048
// back to bf16 16 us (0.94).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/situ_fp8.h"
#include "situ_device.cuh"
#include "situ_fp8.cuh"
#include "situ_host.h"

namespace {

using namespace situ;
using namespace situ_host;
using namespace situ_fp8;

// 8 consecutive elements of a lane, as loaded: 16 bytes of bf16 or 32 of fp32.
template <bool F32>
using Chunk = Vec<F32 ? 8 : 4>;

template <bool F32>
__device__ __forceinline__ void chunk_values(const Chunk<F32>& c, float (&f)[8]) {
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(c.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(c.w[i]);
            f[2 * i + 1] = bf16_hi(c.w[i]);
        }
    }
}

// The largest magnitude of N chunks; infinities stay, and a NaN wins. Few operations an element: the ALU pipe, not HBM, bounded
// the kernel that looked at each value by itself (65537 x 3584: 130 us).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool F32, int N>
__device__ __forceinline__ float chunks_top(const Chunk<F32> (&c)[N]) {
    if constexpr (F32) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) m = max_nan(m, fabsf(__uint_as_float(c[i].w[k])));
        return m;
    } else {                                 // two bf16 at a time
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(c[i].w[k] & 0x7FFF7FFFu));
        return max_nan(bf16_lo(m), bf16_hi(m));
    }
}

template <bool F32, int N>
__device__ __forceinline__ float chunks_finite_top(const Chunk<F32> (&c)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float f[8];
        chunk_values<F32>(c[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, finite_abs(f[k]));
    }
    return m;
}

__device__ __forceinline__ float halfwarp_max_nan(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ bool is_finite(float a) { return a < __int_as_float(0x7F800000); }   // a >= 0 or NaN

// Codes of a chunk. FINITE: it has no other values.
template <bool F32, bool FINITE>
__device__ __forceinline__ uint2 chunk_codes(const Chunk<F32>& c, float inv) {
    float f[8];
    chunk_values<F32>(c, f);
    if constexpr (FINITE) {
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = e4m3x2_from_f32(f[2 * k] * inv, f[2 * k + 1] * inv);
        return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    } else {
        return encode8(f, inv);
    }
}

template <bool F32>
__device__ __forceinline__ float load_one(const void* x, int64_t i) {
    if constexpr (F32) return __ldg((const float*)x + i);
    else return bf16_to_f32(__ldg((const uint16_t*)x + i));
}

template <bool F32>
__device__ __forceinline__ void store_one(void* x, int64_t i, float v) {
    if constexpr (F32) ((float*)x)[i] = v;
    else ((uint16_t*)x)[i] = f32_to_bf16(v);
}

// ---------------------------------------------------------------- rows

// Vector path: D % 8 == 0. A lane takes 8 elements, half a warp a block; a warp takes U steps of 256 elements at once, all
// loaded before any is used. cpr chunks of 8 a row, nb blocks; rows whose D is a multiple of 128 come as one
// long row, for no block straddles two of them.
template <bool F32, int U, int TPB>
__global__ void __launch_bounds__(TPB)
    quant_rows_kernel(const Chunk<F32>* __restrict__ x, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                      int64_t rows, int64_t cpr, int64_t nb, int64_t pieces) {
    let_dependents_go();                     // a product usually follows: its launch and setup run beside this kernel's end
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (TPB / 32), items = rows * pieces;
    for (int64_t it = (int64_t)blockIdx.x * (TPB / 32) + (threadIdx.x >> 5); it < items; it += warps) {
        const int64_t r = rows == 1 ? 0 : it / pieces;
        const int64_t c0 = (it - r * pieces) * (32 * U) + lane;
        const Chunk<F32>* xr = x + r * cpr;
        Chunk<F32> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + 32 * u < cpr) {
                v[u] = ld_stream<F32 ? 8 : 4, true>(xr + c0 + 32 * u);
            } else {
#pragma unroll
                for (int i = 0; i < (F32 ? 8 : 4); ++i) v[u].w[i] = 0u;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + 32 * u;
            float top = halfwarp_max_nan(chunks_top<F32, 1>({v[u]}));
            const bool finite = __all_sync(0xffffffffu, is_finite(top));
            if (!finite) top = halfwarp_max(chunks_finite_top<F32, 1>({v[u]}));
            const int b = scale_byte(top);
            const float inv = inverse_scale(b);
            if (c < cpr) {
                codes[r * cpr + c] = finite ? chunk_codes<F32, true>(v[u], inv) : chunk_codes<F32, false>(v[u], inv);
                if ((lane & 15) == 0) scales[r * nb + (c >> 4)] = (uint8_t)b;
            }
        }
    }
}

// Any D and alignment: a warp a block, lane l elements l, l + 32, ..
template <bool F32>
__global__ void __launch_bounds__(256)
    quant_rows_any_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                          int64_t rows, int64_t D, int64_t nb) {
    let_dependents_go();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * 8, items = rows * nb;
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += warps) {
        const int64_t r = it / nb, c0 = (it - r * nb) * QBLOCK + lane;
        float f[4], m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = c0 + 32 * i < D ? load_one<F32>(x, r * D + c0 + 32 * i) : 0.0f;
            m = fmaxf(m, finite_abs(f[i]));
        }
        const int b = scale_byte(warp_max(m));
        const float inv = inverse_scale(b);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + 32 * i < D) codes[r * D + c0 + 32 * i] = (uint8_t)encode2(f[i], 0.0f, inv);
        if (lane == 0) scales[it] = (uint8_t)b;
    }
}

// ---------------------------------------------------------------- weights: blocks of 128 x 128

// The largest of the block's WARPS warps, of values at least 0; a NaN wins.
template <int WARPS>
__device__ __forceinline__ float block_max(float m, float* shared) {
    m = halfwarp_max_nan(m);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = m;
    __syncthreads();
    m = shared[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) m = max_nan(m, shared[i]);
    __syncthreads();                         // shared may be written again
    return m;
}

// A block of threads per 128 x 128 tile, which stays in registers between the maximum and the codes: 8 elements of 8 rows (bf16)
// or 4 (fp32: 64 registers a thread, 103 with 8 rows) a thread (D % 8 == 0).
template <bool F32>
constexpr int TILE_ROWS = F32 ? 4 : 8;
template <bool F32>
constexpr int TILE_TPB = 2048 / TILE_ROWS<F32>;

template <bool F32>
__global__ void __launch_bounds__(TILE_TPB<F32>, F32 ? 2 : 3)
    quant_tiles_kernel(const Chunk<F32>* __restrict__ x, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                       int64_t tiles, int64_t R, int64_t cpr, int64_t rb, int64_t nb) {
    constexpr int N = TILE_ROWS<F32>, ROWS = 128 / N, WARPS = TILE_TPB<F32> / 32;
    __shared__ float shared[WARPS];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t er = t / nb, e = er / rb;
        const int64_t c = (t - er * nb) * 16 + col, r0 = (er - e * rb) * QBLOCK + row;
        const int64_t at = (e * R + r0) * cpr + c;
        Chunk<F32> v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (c < cpr && r0 + ROWS * i < R) {
                v[i] = ld_stream<F32 ? 8 : 4, true>(x + at + ROWS * i * cpr);
            } else {
#pragma unroll
                for (int k = 0; k < (F32 ? 8 : 4); ++k) v[i].w[k] = 0u;
            }
        }
        float top = block_max<WARPS>(chunks_top<F32>(v), shared);
        const bool finite = is_finite(top);  // the same for all threads
        if (!finite) top = block_max<WARPS>(chunks_finite_top<F32>(v), shared);
        const int b = scale_byte(top);
        const float inv = inverse_scale(b);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c < cpr && r0 + ROWS * i < R)
                codes[at + ROWS * i * cpr] = finite ? chunk_codes<F32, true>(v[i], inv) : chunk_codes<F32, false>(v[i], inv);
        if (threadIdx.x == 0) scales[t] = (uint8_t)b;
    }
}

// Any D and alignment: two passes over the tile.
template <bool F32>
__global__ void __launch_bounds__(256)
    quant_tiles_any_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                           int64_t tiles, int64_t R, int64_t D, int64_t rb, int64_t nb) {
    __shared__ float shared[8];
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t er = t / nb, e = er / rb;
        const int64_t c = (t - er * nb) * QBLOCK + (threadIdx.x & 127), r0 = (er - e * rb) * QBLOCK;
        const int64_t r1 = r0 + QBLOCK < R ? r0 + QBLOCK : R;
        float m = 0.0f;
        if (c < D)
            for (int64_t r = r0 + (threadIdx.x >> 7); r < r1; r += 2) m = fmaxf(m, finite_abs(load_one<F32>(x, (e * R + r) * D + c)));
        const int b = scale_byte(block_max<8>(m, shared));
        const float inv = inverse_scale(b);
        if (c < D)
            for (int64_t r = r0 + (threadIdx.x >> 7); r < r1; r += 2) {
                const int64_t i = (e * R + r) * D + c;
                codes[i] = (uint8_t)encode2(load_one<F32>(x, i), 0.0f, inv);
            }
        if (threadIdx.x == 0) scales[t] = (uint8_t)b;
    }
}

// ---------------------------------------------------------------- back

// 8 codes a lane (D % 8 == 0), rows and weights alike: the scale of element (e, r, d) is
// scales[(e·rb + r / block_rows)·nb + d / 128]. FLAT: rows whose D is a multiple of 128, so chunk i has scale i / 16.
template <bool F32, bool FLAT>
__global__ void __launch_bounds__(256)
    dequant_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, Chunk<F32>* __restrict__ x,
                   int64_t chunks, int64_t R, int64_t cpr, int64_t rb, int64_t nb, int block_shift) {
    constexpr int U = 4;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < chunks; i0 += step * U) {
        uint2 q[U];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * step;
            if (i < chunks) {
                asm("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(q[u].x), "=r"(q[u].y) : "l"(codes + i));
                int64_t at = i >> 4;
                if constexpr (!FLAT) {
                    const int64_t er = i / cpr, c = i - er * cpr;
                    at = er;                 // the scales' row
                    if (block_shift) {
                        const int64_t e = er / R;
                        at = e * rb + ((er - e * R) >> block_shift);
                    }
                    at = at * nb + (c >> 4);
                }
                s[u] = scale_value(__ldg(scales + at));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * step;
            if (i >= chunks) break;
            float f[8];
            decode8(q[u], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= s[u];
            Chunk<F32> v;
            if constexpr (F32) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v.w[k] = __float_as_uint(f[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v.w[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
            }
            st_stream<F32 ? 8 : 4>(x + i, v);
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(256)
    dequant_any_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, void* __restrict__ x,
                       int64_t n, int64_t R, int64_t D, int64_t rb, int64_t nb, int block_shift) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const int64_t er = i / D, c = i - er * D, e = er / R;
        const int64_t at = e * rb + ((er - e * R) >> block_shift);
        float lo, hi;
        e4m3x2_to_f32(codes[i], lo, hi);
        store_one<F32>(x, i, lo * scale_value(scales[at * nb + c / QBLOCK]));
    }
}

// ---------------------------------------------------------------- host side

constexpr int ROWS_TPB = 256;
constexpr int64_t FEW_CHUNKS = 1 << 18;      // of 8 elements

template <bool F32>
int launch_quant(const void* x, uint8_t* codes, uint8_t* scales, int64_t E, int64_t R, int64_t D, int block_rows,
                 cudaStream_t stream) {
    const bool vec = D % 8 == 0 && aligned(x, F32 ? 32 : 16) && aligned(codes, 8);
    const int64_t nb = (D + QBLOCK - 1) / QBLOCK;
    if (block_rows == 1) {
        int64_t rows = E * R;
        if (!vec) return launch(quant_rows_any_kernel<F32>, 256, rows * nb, stream, x, codes, scales, rows, D, nb);
        int64_t cpr = D / 8;
        if (D % QBLOCK == 0) {
            cpr *= rows;
            rows = 1;
        }
        constexpr int U = F32 ? 2 : 4;
        const auto go = [&](auto kernel, int u) {
            const int64_t pieces = (cpr + 32 * u - 1) / (32 * u);
            return launch(kernel, ROWS_TPB, rows * pieces, stream, (const Chunk<F32>*)x, (uint2*)codes, scales, rows, cpr,
                          nb, pieces);
        };
        // Few elements: one step a warp, over as many SMs as there are (one step / U steps, us, bf16 rows of 3584: 8 rows 1.4 /
        // 2.2, 256 rows 1.9 / 2.3, 512 rows 2.5 / 2.6, 1024 rows 3.4 / 3.0, 16384 rows 34.5 / 26.2; fp32 the same way).
        // Measured of rows that run together; where D is no multiple of 128 a warp's U steps end with its row, and short rows
        // leave most of them empty: bf16 262144 x 144 85 us (0.20 of the copy rate; fp32, U = 2, 64 us), 1048576 x 16 308 us
        // (0.03), 65537 x 1008 40 us (0.75).
        return rows * cpr <= FEW_CHUNKS ? go(quant_rows_kernel<F32, 1, ROWS_TPB>, 1) : go(quant_rows_kernel<F32, U, ROWS_TPB>, U);
    }
    const int64_t rb = (R + QBLOCK - 1) / QBLOCK, tiles = E * rb * nb;
    if (!vec) return launch(quant_tiles_any_kernel<F32>, 256, tiles * 8, stream, x, codes, scales, tiles, R, D, rb, nb);
    return launch(quant_tiles_kernel<F32>, TILE_TPB<F32>, tiles * (TILE_TPB<F32> / 32), stream, (const Chunk<F32>*)x, (uint2*)codes, scales, tiles, R,
                  D / 8, rb, nb);
}

template <bool F32>
int launch_dequant(const uint8_t* codes, const uint8_t* scales, void* x, int64_t E, int64_t R, int64_t D, int block_rows,
                   cudaStream_t stream) {
    const int64_t nb = (D + QBLOCK - 1) / QBLOCK, rb = (R + block_rows - 1) / block_rows;
    const int shift = block_rows == 1 ? 0 : 7;
    if (D % 8 == 0 && aligned(x, F32 ? 32 : 16) && aligned(codes, 8)) {
        const int64_t chunks = E * R * (D / 8);
        return launch(block_rows == 1 && D % QBLOCK == 0 ? dequant_kernel<F32, true> : dequant_kernel<F32, false>, 256, (chunks + 31) / 32, stream, (const uint2*)codes, scales, (Chunk<F32>*)x,
                      chunks, R, D / 8, rb, nb, shift);
    }
    return launch(dequant_any_kernel<F32>, 256, (E * R * D + 31) / 32, stream, codes, scales, x, E * R * D, R, D, rb, nb,
                  shift);
}

int check_blocks(int type, int64_t E, int64_t R, int64_t D, int block_rows) {
    if ((type != SITU_BF16 && type != SITU_FP32) || E < 0 || R < 0 || D < 1 || (block_rows != 1 && block_rows != QBLOCK))
        return SITU_GLU_INVALID_ARG;
    const int64_t most = (int64_t)1 << 62;
    if (D >= most || R >= most / D || (R && E >= most / D / R)) return SITU_GLU_INVALID_ARG;
    return SITU_GLU_OK;
}

int check_buffers(const void* x, int type, const void* codes, const void* scales, int64_t E, int64_t R, int64_t D,
                  int block_rows, bool into_x) {
    if (!x || !codes || !scales || !aligned(x, type == SITU_FP32 ? 4 : 2)) return SITU_GLU_INVALID_ARG;
    const int64_t n = E * R * D;
    const Range rx = range_of(x, n * (type == SITU_FP32 ? 4 : 2)), rc = range_of(codes, n);
    const Range rs = range_of(scales, E * ((R + block_rows - 1) / block_rows) * ((D + QBLOCK - 1) / QBLOCK));
    if (overlap(rx, rc) || overlap(rx, rs) || (!into_x && overlap(rc, rs))) return SITU_GLU_OVERLAP;
    return SITU_GLU_OK;
}

}  // namespace

extern "C" {

int situ_quant_fp8(const void* x, int type, uint8_t* codes, uint8_t* scales, int64_t E, int64_t R, int64_t D,
                   int block_rows, cudaStream_t stream) {
    int st = check_blocks(type, E, R, D, block_rows);
    if (st != SITU_GLU_OK || E == 0 || R == 0) return st;
    st = check_buffers(x, type, codes, scales, E, R, D, block_rows, false);
    if (st != SITU_GLU_OK) return st;
    return type == SITU_FP32 ? launch_quant<true>(x, codes, scales, E, R, D, block_rows, stream)
                             : launch_quant<false>(x, codes, scales, E, R, D, block_rows, stream);
}

int situ_dequant_fp8(const uint8_t* codes, const uint8_t* scales, void* x, int type, int64_t E, int64_t R, int64_t D,
                     int block_rows, cudaStream_t stream) {
    int st = check_blocks(type, E, R, D, block_rows);
    if (st != SITU_GLU_OK || E == 0 || R == 0) return st;
    st = check_buffers(x, type, codes, scales, E, R, D, block_rows, true);
    if (st != SITU_GLU_OK) return st;
    return type == SITU_FP32 ? launch_dequant<true>(codes, scales, x, E, R, D, block_rows, stream)
                             : launch_dequant<false>(codes, scales, x, E, R, D, block_rows, stream);
}

}  // extern "C"
