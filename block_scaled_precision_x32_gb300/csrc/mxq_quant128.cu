// mxq_quant128.cu -- activations and gradients to E4M3 with one power-of-two
// scale per 128 elements, along the rows (1x128) or down the columns (128x1).
//
// For a block with largest magnitude amax = (1 + f) 2^E the scale is the
// least power of two that keeps amax / 2^s within E4M3's largest value
// 448 = 1.75 * 2^8: s = E - 8, and one more if f > 0.75.
#include <cuda_bf16.h>

#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

// UE8M0 code of a block from the bits of its fp32 amax; 255 for NaN and Inf.
__device__ __forceinline__ uint32_t scale_code128(uint32_t amax) {
    const int E = (int)(amax >> 23);
    if (E == 255) return 255u;
    const int s = E - 135 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(max(s, -127) + 127);  // s <= 120: no upper clamp is reached
}

// 2^-s for a code below 255: s in [-127, 120].
__device__ __forceinline__ uint32_t inv_scale128(uint32_t code) { return (254u - code) << 23; }

template <Elt ELT>
__device__ __forceinline__ uint32_t load_f32(const void* x, int64_t i) {
    if constexpr (ELT == Elt::BF16) return (uint32_t)static_cast<const uint16_t*>(x)[i] << 16;
    return static_cast<const uint32_t*>(x)[i];
}

// Source row of output row r, -1 for a row of zeros.
__device__ __forceinline__ int64_t source_row(const Quant128Args& a, int64_t r) {
    if (!a.index) return r;
    const int32_t i = a.index[r];
    const int64_t t = i < 0 ? -1 : i / a.index_div;
    return t < a.rows ? t : -1;
}

// One warp per 1x128 block.
template <Elt ELT>
__global__ void __launch_bounds__(256) quant_rows_kernel(Quant128Args a, int64_t nb) {
    const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 32;
    if (unit >= a.out_rows * nb) return;
    const int64_t r = unit / nb, b = unit - r * nb;
    const int lane = threadIdx.x & 31;
    const int64_t src = source_row(a, r);
    const int64_t k0 = b * 128 + lane * 4;
    uint32_t v[4];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = src >= 0 && k0 + i < a.K ? load_f32<ELT>(a.x, src * a.ldx + k0 + i) : 0u;
        amax = max(amax, v[i] & 0x7FFFFFFFu);
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    const uint32_t code = scale_code128(amax);
    if (lane == 0) a.scales[r * nb + b] = (uint8_t)code;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k0 + i < a.K)
            a.data[r * a.K + k0 + i] =
                code == 255u ? 0x7F : (uint8_t)e4m3x2_from_f32(0u, f32_mul(v[i], inv_scale128(code)));
}

// One thread per 128x1 block.
template <Elt ELT>
__global__ void __launch_bounds__(128) quant_columns_kernel(Quant128Args a) {
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (c >= a.K) return;
    const int64_t r0 = (int64_t)blockIdx.y * 128, r1 = min(r0 + 128, a.out_rows);
    uint32_t amax = 0;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t src = source_row(a, r);
        if (src >= 0) amax = max(amax, load_f32<ELT>(a.x, src * a.ldx + c) & 0x7FFFFFFFu);
    }
    const uint32_t code = scale_code128(amax);
    a.scales[(int64_t)blockIdx.y * a.K + c] = (uint8_t)code;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t src = source_row(a, r);
        const uint32_t v = src >= 0 ? load_f32<ELT>(a.x, src * a.ldx + c) : 0u;
        a.data[r * a.K + c] = code == 255u ? 0x7F : (uint8_t)e4m3x2_from_f32(0u, f32_mul(v, inv_scale128(code)));
    }
}

template <Elt ELT>
cudaError_t launch(bool columns, const Quant128Args& a, cudaStream_t s) {
    if (columns) {
        // blockIdx.y reaches 65535: 2^23 rows at a time
        for (int64_t r0 = 0; r0 < a.out_rows; r0 += INT64_C(128) * 65535) {
            Quant128Args p = a;
            p.out_rows = a.out_rows - r0 < INT64_C(128) * 65535 ? a.out_rows - r0 : INT64_C(128) * 65535;
            if (a.index) {
                p.index = a.index + r0;
            } else {
                p.x = static_cast<const char*>(a.x) + r0 * a.ldx * (ELT == Elt::BF16 ? 2 : 4);
                p.rows = p.out_rows;
            }
            p.data = a.data + r0 * a.K;
            p.scales = a.scales + r0 / 128 * a.K;
            quant_columns_kernel<ELT>
                <<<dim3((unsigned)ceil_div(a.K, 128), (unsigned)ceil_div(p.out_rows, 128)), 128, 0, s>>>(p);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    const int64_t nb = ceil_div(a.K, 128);
    if (ceil_div(a.out_rows * nb, 8) > INT64_C(0x7FFFFFFF)) return cudaErrorInvalidValue;
    quant_rows_kernel<ELT><<<(unsigned)ceil_div(a.out_rows * nb, 8), 256, 0, s>>>(a, nb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant128(Elt elt, bool columns, const Quant128Args& a, cudaStream_t s) {
    return elt == Elt::BF16 ? launch<Elt::BF16>(columns, a, s) : launch<Elt::FP32>(columns, a, s);
}

}  // namespace mxq
