// mxq_quant128.cu -- activations and gradients to E4M3 with one power-of-two
// scale per 128 elements, along the rows (1x128) or down the columns (128x1).
//
// For a block with largest magnitude amax = (1 + f) 2^E the scale is the
// least power of two that keeps amax / 2^s within E4M3's largest value
// 448 = 1.75 * 2^8: s = E - 8, and one more if f > 0.75.
#include <cuda_bf16.h>

#include "mxq_device.cuh"
#include "mxq_layer.h"
#include "mxq_launch.cuh"

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

// 16 consecutive elements as fp32 patterns, 32-byte loads.
template <Elt ELT>
struct Unit {
    uint32_t w[ELT == Elt::BF16 ? 8 : 16];

    __device__ __forceinline__ void load(const void* x, int64_t i) {
        if constexpr (ELT == Elt::BF16) {
            ld32(w, static_cast<const uint16_t*>(x) + i);
        } else {
            ld32(reinterpret_cast<uint32_t(&)[8]>(w[0]), static_cast<const uint32_t*>(x) + i);
            ld32(reinterpret_cast<uint32_t(&)[8]>(w[8]), static_cast<const uint32_t*>(x) + i + 8);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& v : w) v = 0;
    }
    __device__ __forceinline__ uint32_t at(int i) const {
        if constexpr (ELT == Elt::BF16) return i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16;
        return w[i];
    }
};

// Rows of 16-element units, eight lanes to a 1x128 block: 32 bytes (bf16) or
// 64 (fp32) of loads and one 16-byte store a lane, the block's maximum by
// three shuffles.  Memory-bound: one unit a thread, so that registers leave
// room for as many threads as there can be (8192 x 7184 bf16: 29.6 us, 5.98
// TB/s; two units 31.7, four 34.8; fp32 42.7 us, 6.9 TB/s).  Gathered rows are
// read and rounded once for each choice: 8191 x 4 of 7184 bf16 123 us.
template <Elt ELT>
__global__ void __launch_bounds__(256) quant_rows_unit_kernel(Quant128Args a, int64_t nb) {
    let_next_start();
    wait_for_stream();
    const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x, total = a.out_rows * nb * 8;
    int64_t row, b;
    split_index(unit >> 3, nb, row, b);
    const int64_t k = b * 128 + (threadIdx.x & 7) * 16;
    const int64_t src = unit < total && k < a.K ? source_row(a, row) : -1;
    Unit<ELT> u;
    if (src >= 0)
        u.load(a.x, src * a.ldx + k);
    else
        u.clear();
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = max(amax, u.at(j) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    const uint32_t code = scale_code128(amax), inv = inv_scale128(code);
    if (unit >= total) return;
    if ((threadIdx.x & 7) == 0) a.scales[row * nb + b] = (uint8_t)code;
    if (k >= a.K) return;
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        o[j] = e4m3x2_from_f32(f32_mul(u.at(4 * j + 1), inv), f32_mul(u.at(4 * j), inv)) |
               e4m3x2_from_f32(f32_mul(u.at(4 * j + 3), inv), f32_mul(u.at(4 * j + 2), inv)) << 16;
        if (code == 255u) o[j] = 0x7F7F7F7Fu;
    }
    st16(a.data + row * a.K + k, o[0], o[1], o[2], o[3]);
}

// Any alignment and any K: a warp per four 1x128 blocks, an element at a time,
// neighbours to neighbouring lanes; the loads of all four are on their way at
// once.  Bound by instructions, one load and one byte store an element: 4095 x
// 7183 46 us as bf16, 36 as fp32 (4.1 TB/s).
template <Elt ELT>
__global__ void __launch_bounds__(256) quant_rows_kernel(Quant128Args a, int64_t nb) {
    let_next_start();
    wait_for_stream();
    constexpr int B = 4;
    const int64_t first = ((int64_t)blockIdx.x * 8 + threadIdx.x / 32) * B;
    const int lane = threadIdx.x & 31;
    uint32_t v[B][4];
    int64_t row[B], k0[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        split_index(first + i, nb, row[i], k0[i]);
        k0[i] = k0[i] * 128 + lane;
        const int64_t src = row[i] < a.out_rows ? source_row(a, row[i]) : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[i][j] = src >= 0 && k0[i] + 32 * j < a.K ? load_f32<ELT>(a.x, src * a.ldx + k0[i] + 32 * j) : 0u;
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = max(amax, v[i][j] & 0x7FFFFFFFu);
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        if (row[i] >= a.out_rows) break;
        const uint32_t code = scale_code128(amax);
        if (lane == 0) a.scales[first + i] = (uint8_t)code;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k0[i] + 32 * j < a.K)
                a.data[row[i] * a.K + k0[i] + 32 * j] =
                    code == 255u ? 0x7F : (uint8_t)e4m3x2_from_f32(0u, f32_mul(v[i][j], inv_scale128(code)));
    }
}

// Threads along a row, and rows a thread (bytes in flight are alike).
template <Elt ELT>
struct ColumnTile {
    static constexpr int kX = 4, kRows = ELT == Elt::BF16 ? 8 : 4;
    static constexpr int kY = 128 / kRows, kThreads = kX * kY;
};

// 128 rows x 32 columns a block, 8 columns of 4 (fp32) or 8 rows a thread, all
// in registers between the maximum and the rounding: each element is read
// once.  The maximum of a column goes through shuffles among the threads of a
// warp that share it, and shared memory.  4099 x 4096 fp32: 14.8 us, 5.7 TB/s
// (wider and narrower blocks 1 to 3 us more; one thread a column, reading
// twice, 44), 8191 x 7184 bf16: 33.3 us, 5.3 TB/s: held back by the two
// barriers of a block, the last wave of blocks and, for bf16, arithmetic.
template <Elt ELT>
__global__ void __launch_bounds__(ColumnTile<ELT>::kThreads) quant_columns_tile_kernel(Quant128Args a) {
    let_next_start();
    wait_for_stream();
    constexpr int R = ColumnTile<ELT>::kRows, TX = ColumnTile<ELT>::kX, TY = ColumnTile<ELT>::kY, WARPS = TX * TY / 32;
    __shared__ uint4 top[WARPS][2 * TX];  // [warp][columns]
    __shared__ uint2 codes[TX];        // a byte a column
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int64_t c = ((int64_t)blockIdx.x * TX + tx) * 8, r0 = (int64_t)blockIdx.y * 128 + ty;
    uint32_t v[R][ELT == Elt::BF16 ? 4 : 8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + TY * i;
        const int64_t src = r < a.out_rows && c < a.K ? source_row(a, r) : -1;
#pragma unroll
        for (uint32_t& x : v[i]) x = 0;
        if (src >= 0) {
            if constexpr (ELT == Elt::BF16) {
                const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + src * a.ldx + c);
                v[i][0] = q.x, v[i][1] = q.y, v[i][2] = q.z, v[i][3] = q.w;
            } else {
                ld32(v[i], static_cast<const uint32_t*>(a.x) + src * a.ldx + c);
            }
        }
    }
    const auto at = [&](int i, int j) {
        if constexpr (ELT == Elt::BF16) return j & 1 ? v[i][j / 2] & 0xFFFF0000u : v[i][j / 2] << 16;
        else return v[i][j];
    };
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) m[j] = max(m[j], at(i, j) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = TX; d < 32; d *= 2) m[j] = max(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], d));
    }
    if ((threadIdx.x & 31) < TX) {
        top[threadIdx.x / 32][2 * tx] = make_uint4(m[0], m[1], m[2], m[3]);
        top[threadIdx.x / 32][2 * tx + 1] = make_uint4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    if (threadIdx.x < 8 * TX) {
        uint32_t amax = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) amax = max(amax, reinterpret_cast<const uint32_t*>(top[w])[threadIdx.x]);
        const uint8_t own = (uint8_t)scale_code128(amax);
        reinterpret_cast<uint8_t*>(codes)[threadIdx.x] = own;
        const int64_t column = (int64_t)blockIdx.x * (8 * TX) + threadIdx.x;
        if (column < a.K) a.scales[(int64_t)blockIdx.y * a.K + column] = own;
    }
    __syncthreads();
    if (c >= a.K) return;
    uint32_t inv[8], nan[2] = {};  // nan: bytes of poisoned columns
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t code = ((j < 4 ? codes[tx].x : codes[tx].y) >> (8 * (j & 3))) & 0xFFu;
        inv[j] = inv_scale128(code);
        nan[j / 4] |= code == 255u ? 0xFFu << (8 * (j & 3)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (r0 + TY * i >= a.out_rows) break;
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = 4 * h;
            const uint32_t lo = e4m3x2_from_f32(f32_mul(at(i, j + 1), inv[j + 1]), f32_mul(at(i, j), inv[j])),
                           hi = e4m3x2_from_f32(f32_mul(at(i, j + 3), inv[j + 3]), f32_mul(at(i, j + 2), inv[j + 2]));
            o[h] = lop_select(0x7F7F7F7Fu, lo | hi << 16, nan[h]);
        }
        *reinterpret_cast<uint2*>(a.data + (r0 + TY * i) * a.K + c) = make_uint2(o[0], o[1]);
    }
}

// Any alignment and any K: 128 rows x 64 columns a block, 16 rows of one column
// a thread, an element at a time: 4095 x 7183 fp32 46 us, 3.2 TB/s.
template <Elt ELT>
__global__ void __launch_bounds__(512) quant_columns_kernel(Quant128Args a) {
    let_next_start();
    wait_for_stream();
    constexpr int R = 16, Y = 8;
    __shared__ uint32_t top[Y][64];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + tx, r0 = (int64_t)blockIdx.y * 128 + ty;
    uint32_t v[R], amax = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + Y * i;
        const int64_t src = r < a.out_rows && c < a.K ? source_row(a, r) : -1;
        v[i] = src >= 0 ? load_f32<ELT>(a.x, src * a.ldx + c) : 0u;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) amax = max(amax, v[i] & 0x7FFFFFFFu);
    top[ty][tx] = amax;
    __syncthreads();
    if (c >= a.K) return;
#pragma unroll
    for (int y = 0; y < Y; ++y) amax = max(amax, top[y][tx]);
    const uint32_t code = scale_code128(amax);
    if (ty == 0) a.scales[(int64_t)blockIdx.y * a.K + c] = (uint8_t)code;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (r0 + Y * i < a.out_rows)
            a.data[(r0 + Y * i) * a.K + c] =
                code == 255u ? 0x7F : (uint8_t)e4m3x2_from_f32(0u, f32_mul(v[i], inv_scale128(code)));
}

bool on(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <Elt ELT>
cudaError_t launch(bool columns, const Quant128Args& a, cudaStream_t s) {
    constexpr int64_t es = ELT == Elt::BF16 ? 2 : 4;
    const bool one_row = a.rows <= 1;  // then the stride is not used
    if (columns) {
        // 8 columns: 16 bytes of bf16, 32 of fp32, 8 of payload and scales
        const bool tiled = a.K % 8 == 0 && on(a.x, 8 * es) && (one_row || a.ldx * es % (8 * es) == 0) && on(a.data, 8) &&
                           on(a.scales, 8);
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
            const unsigned y = (unsigned)ceil_div(p.out_rows, 128);
            const cudaError_t e =
                tiled ? launch_overlapped(quant_columns_tile_kernel<ELT>, dim3((unsigned)ceil_div(a.K, 8 * ColumnTile<ELT>::kX), y),
                                          ColumnTile<ELT>::kThreads, 0, 0, s, p)
                      : launch_overlapped(quant_columns_kernel<ELT>, dim3((unsigned)ceil_div(a.K, 64), y), 512, 0, 0, s, p);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    const int64_t nb = ceil_div(a.K, 128);
    if (ceil_div(a.out_rows * nb, 8) > INT64_C(0x7FFFFFFF)) return cudaErrorInvalidValue;  // over 2 TB of elements
    // units of 16 elements: 32-byte loads and 16-byte stores
    if (a.K % 16 == 0 && on(a.x, 32) && (one_row || a.ldx * es % 32 == 0) && on(a.data, 16)) {
        return launch_overlapped(quant_rows_unit_kernel<ELT>, dim3((unsigned)ceil_div(a.out_rows * nb * 8, 256)), 256, 0, 0, s, a,
                                 nb);
    }
    return launch_overlapped(quant_rows_kernel<ELT>, dim3((unsigned)ceil_div(a.out_rows * nb, 32)), 256, 0, 0, s, a, nb);
}

}  // namespace

cudaError_t launch_quant128(Elt elt, bool columns, const Quant128Args& a, cudaStream_t s) {
    const cudaError_t e = elt == Elt::BF16 ? launch<Elt::BF16>(columns, a, s) : launch<Elt::FP32>(columns, a, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace mxq
