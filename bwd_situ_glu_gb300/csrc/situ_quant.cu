// situ_quant.cu — block-scaled quantisation to E4M3 with power-of-two scales, and back (include/situ_fp8.h).
//
// A block's scale is the least power of two that brings its largest finite value to 448 or below. 448 is
// 1.75·2^8, so its exponent follows from the bits of that value alone, and x·2^-e is exact: the code's rounding
// (cvt.rn.satfinite.e4m3x2) is the only one. One read of x, one write of codes; HBM-bound.
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
            float f[8], m = 0.0f;
            chunk_values<F32>(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(f[i]));
            const int b = scale_byte(halfwarp_max(m));
            const int64_t c = c0 + 32 * u;
            if (c < cpr) {
                codes[r * cpr + c] = encode8(f, inverse_scale(b));
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

// The largest of the block's threads (256).
__device__ __forceinline__ float block_max(float m, float* shared) {
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = m;
    __syncthreads();
    m = shared[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, shared[i]);
    __syncthreads();                         // shared may be written again
    return m;
}

// A block of threads per 128 x 128 tile, which stays in registers between the maximum and the codes: 8 elements of 8 rows a
// thread (D % 8 == 0).
template <bool F32>
__global__ void __launch_bounds__(256)
    quant_tiles_kernel(const Chunk<F32>* __restrict__ x, uint2* __restrict__ codes, uint8_t* __restrict__ scales,
                       int64_t tiles, int64_t R, int64_t cpr, int64_t rb, int64_t nb) {
    __shared__ float shared[8];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t er = t / nb, e = er / rb;
        const int64_t c = (t - er * nb) * 16 + col, r0 = (er - e * rb) * QBLOCK + row;
        const int64_t at = (e * R + r0) * cpr + c;
        Chunk<F32> v[8];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c < cpr && r0 + 16 * i < R) {
                v[i] = ld_stream<F32 ? 8 : 4, true>(x + at + 16 * i * cpr);
            } else {
#pragma unroll
                for (int k = 0; k < (F32 ? 8 : 4); ++k) v[i].w[k] = 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            chunk_values<F32>(v[i], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, finite_abs(f[k]));
        }
        const int b = scale_byte(block_max(m, shared));
        const float inv = inverse_scale(b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f[8];
            chunk_values<F32>(v[i], f);
            if (c < cpr && r0 + 16 * i < R) codes[at + 16 * i * cpr] = encode8(f, inv);
        }
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
        const int b = scale_byte(block_max(m, shared));
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
// scales[(e·rb + r / block_rows)·nb + d / 128].
template <bool F32>
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
                const int64_t er = i / cpr, c = i - er * cpr;
                int64_t at = er;             // the scales' row
                if (block_shift) {
                    const int64_t e = er / R;
                    at = e * rb + ((er - e * R) >> block_shift);
                }
                s[u] = scale_value(__ldg(scales + at * nb + (c >> 4)));
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
        // few elements: one step a warp, over as many SMs as there are
        return rows * cpr <= 65536 ? go(quant_rows_kernel<F32, 1, ROWS_TPB>, 1) : go(quant_rows_kernel<F32, U, ROWS_TPB>, U);
    }
    const int64_t rb = (R + QBLOCK - 1) / QBLOCK, tiles = E * rb * nb;
    if (!vec) return launch(quant_tiles_any_kernel<F32>, 256, tiles * 8, stream, x, codes, scales, tiles, R, D, rb, nb);
    return launch(quant_tiles_kernel<F32>, 256, tiles * 8, stream, (const Chunk<F32>*)x, (uint2*)codes, scales, tiles, R,
                  D / 8, rb, nb);
}

template <bool F32>
int launch_dequant(const uint8_t* codes, const uint8_t* scales, void* x, int64_t E, int64_t R, int64_t D, int block_rows,
                   cudaStream_t stream) {
    const int64_t nb = (D + QBLOCK - 1) / QBLOCK, rb = (R + block_rows - 1) / block_rows;
    const int shift = block_rows == 1 ? 0 : 7;
    if (D % 8 == 0 && aligned(x, F32 ? 32 : 16) && aligned(codes, 8)) {
        const int64_t chunks = E * R * (D / 8);
        return launch(dequant_kernel<F32>, 256, (chunks + 31) / 32, stream, (const uint2*)codes, scales, (Chunk<F32>*)x,
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
