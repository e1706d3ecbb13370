// mxq_matmul.cu -- products of block-scaled FP8 operands:
//   out[i, j] = sum_b 2^(sa(i, b) + sb(j, b)) sum_{k in block b} A[i, k] B[j, k]
// with blocks of 128 along the depth, accumulated in fp32.
#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kNaNScale = 1 << 20;

// Exponent of the scale of row i and depth block kb.
__device__ __forceinline__ int operand_scale(const MatOperand& o, int64_t e, int64_t i, int64_t kb) {
    if (o.tiles) {
        const uint32_t t = static_cast<const uint32_t*>(o.scales)[e * o.s_expert + (i >> 7) * o.s_row + kb * o.s_kb];
        if (t == 0x00400000u) return -127;
        const bool power = (t & 0x7FFFFFu) == 0u && t - 1u < 0x7F7FFFFFu;
        return power ? (int)(t >> 23) - 127 : kNaNScale;
    }
    const int c = static_cast<const uint8_t*>(o.scales)[i * o.s_row + kb * o.s_kb];
    return c == 255 ? kNaNScale : c - 127;
}

__device__ __forceinline__ float operand_value(const MatOperand& o, int64_t e, int64_t i, int64_t k) {
    const uint8_t* at = o.data + e * o.expert + (o.mn ? k * o.ld + i : i * o.ld + k);
    return __uint_as_float(decode_scaled<false>(*at, 0x3F800000u));
}

// v * 2^e
__device__ __forceinline__ float times_power(float v, int e) {
    if (e >= kNaNScale / 2) return __uint_as_float(0x7FC00000u);
    const int h = e / 2;  // two powers, each a normal number: |e| <= 254
    return v * __uint_as_float((uint32_t)(h + 127) << 23) * __uint_as_float((uint32_t)(e - h + 127) << 23);
}

__device__ __forceinline__ void store_out(const MatmulArgs& g, int64_t at, float v) {
    uint32_t u = __float_as_uint(v);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0x7FC00000u;
    if (g.out_bf16)
        static_cast<uint16_t*>(g.out)[at] = (uint16_t)bf16_rne(u);
    else
        static_cast<uint32_t*>(g.out)[at] = u;
}

// 64x64 outputs per block of 256 threads, 4x4 each, depth in steps of 16 through shared memory.
__global__ void __launch_bounds__(256) matmul_kernel(MatmulArgs g) {
    __shared__ float As[16][65], Bs[16][65];
    int64_t e = 0, i0 = (int64_t)blockIdx.y * 64, i_end = g.a.rows, k0 = 0, k_end = g.depth, out0 = 0;
    bool zero = false;
    if (g.grouping == Grouping::ROWS) {
        // blocks of 64 rows of the experts in turn; the rows behind the last expert form one more part, of zeros
        int64_t tile = blockIdx.y, lo = 0;
        for (e = 0; e <= g.E; ++e) {
            int64_t hi = e < g.E ? max(lo, min((int64_t)g.offsets[e + 1], g.a.rows)) : g.a.rows;
            if (e == 0) lo = max((int64_t)0, min((int64_t)g.offsets[0], g.a.rows)), hi = max(lo, hi);
            const int64_t n = (hi - lo + 63) / 64;
            if (tile < n) {
                i0 = lo + tile * 64;
                i_end = hi;
                break;
            }
            tile -= n;
            lo = hi;
        }
        if (e > g.E) {  // rows in front of the first expert
            if (tile > 0) return;
            i0 = 0;
            i_end = max((int64_t)0, min((int64_t)g.offsets[0], g.a.rows));
        }
        zero = e >= g.E;
    } else if (g.grouping == Grouping::DEPTH) {
        e = blockIdx.z;
        int64_t lo = 0;
        for (int64_t x = 0; x <= e + 1; ++x) {
            const int64_t v = max(lo, min((int64_t)g.offsets[x], g.depth));
            if (x <= e) k0 = v;
            if (x == e + 1) k_end = v;
            lo = v;
        }
        k0 = (k0 + 127) / 128 * 128;
        out0 = e * g.out_expert;
    }
    const int64_t eb = g.grouping == Grouping::ROWS ? min(e, g.E - 1) : 0;
    for (; i0 < i_end; i0 += zero ? 64 : i_end) {  // zeros: every block of rows in turn, else one
        const int64_t j0 = (int64_t)blockIdx.x * 64;
        const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
        float acc[4][4] = {};
        for (int64_t kb = k0; !zero && kb < k_end; kb = (kb / 128 + 1) * 128) {
            float sum[4][4] = {};
            const int64_t kb_end = min(k_end, (kb / 128 + 1) * 128);
            for (int64_t k = kb; k < kb_end; k += 16) {
                for (int q = threadIdx.x; q < 1024; q += 256) {
                    const int r = q / 16, c = q % 16;
                    As[c][r] = i0 + r < i_end && k + c < kb_end ? operand_value(g.a, 0, i0 + r, k + c) : 0.0f;
                    Bs[c][r] = j0 + r < g.b.rows && k + c < kb_end ? operand_value(g.b, eb, j0 + r, k + c) : 0.0f;
                }
                __syncthreads();
#pragma unroll
                for (int c = 0; c < 16; ++c)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int x = 0; x < 4; ++x) sum[y][x] = fmaf(As[c][ty + 16 * y], Bs[c][tx + 16 * x], sum[y][x]);
                __syncthreads();
            }
            for (int y = 0; y < 4; ++y)
                for (int x = 0; x < 4; ++x) {
                    const int64_t i = i0 + ty + 16 * y, j = j0 + tx + 16 * x;
                    if (i < i_end && j < g.b.rows)
                        acc[y][x] += times_power(sum[y][x], operand_scale(g.a, 0, i, kb >> 7) +
                                                                operand_scale(g.b, eb, j, kb >> 7));
                }
        }
        for (int y = 0; y < 4; ++y)
            for (int x = 0; x < 4; ++x) {
                const int64_t i = i0 + ty + 16 * y, j = j0 + tx + 16 * x;
                if (i < i_end && j < g.b.rows) store_out(g, out0 + i * g.ldo + j, acc[y][x]);
            }
    }
}

__global__ void __launch_bounds__(256) repack_kernel(const uint8_t* src, int64_t ld, int64_t rows, int64_t n,
                                                     uint8_t* dst, int64_t ldd) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * ldd; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / ldd, c = i - r * ldd;
        dst[i] = c < n ? src[r * ld + c] : 0;
    }
}

}  // namespace

cudaError_t launch_matmul(const MatmulArgs& g, cudaStream_t s) {
    dim3 grid((unsigned)ceil_div(g.b.rows, 64), (unsigned)ceil_div(g.a.rows, 64));
    if (g.grouping == Grouping::ROWS) grid.y = (unsigned)(ceil_div(g.a.rows, 64) + g.E + 2);
    if (g.grouping == Grouping::DEPTH) grid.z = (unsigned)g.E;
    if (grid.y > 65535u) return cudaErrorInvalidValue;
    matmul_kernel<<<grid, 256, 0, s>>>(g);
    return cudaGetLastError();
}

cudaError_t launch_repack(const uint8_t* src, int64_t ld, int64_t rows, int64_t n, uint8_t* dst, int64_t ldd,
                          cudaStream_t s) {
    if (rows == 0) return cudaSuccess;
    const int64_t want = ceil_div(rows * ldd, 256);
    const int64_t most = (int64_t)sm_count() * 16;
    repack_kernel<<<(unsigned)(want < most ? want : most), 256, 0, s>>>(src, ld, rows, n, dst, ldd);
    return cudaGetLastError();
}

}  // namespace mxq
