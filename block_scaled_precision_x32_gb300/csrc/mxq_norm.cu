// mxq_norm.cu -- root-mean-square norm of x plus a residual, written as the
// E4M3 operand of the next product (1x128 scales), and its gradient.
//
//   h = RN(x + residual)   r = 1 / sqrt(mean_k h_k^2 + eps)   y_k = (h_k r) w_k
//
// The statistics are those of h as it is stored, so that the gradient, which
// has h alone, is that of what was computed.  y is quantized before it is
// rounded to x's type.  Sums and statistics are fp32.
#include "mxq_device.cuh"
#include "mxq_e4m3.cuh"
#include "mxq_layer.h"
#include "mxq_launch.cuh"

namespace mxq {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d /= 2) v = fadd(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Sum over the block, the same in every thread: lanes, then warps, in a fixed
// order.  `part` is written by this call alone until the block's next barrier.
__device__ __forceinline__ float block_sum(float v, float (&part)[32]) {
    v = warp_sum(v);
    const int warps = blockDim.x / 32;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float sum = 0.0f;
    for (int w = 0; w < warps; ++w) sum = fadd(sum, part[w]);
    return sum;
}

__device__ __forceinline__ float rstd_of(float sum, int64_t K, float eps) {
    return fdiv(1.0f, fsqrt(fadd(fdiv(sum, (float)K), eps)));
}

template <Elt ELT>
__device__ __forceinline__ char* at_row(void* p, int64_t r, int64_t ld) {
    return static_cast<char*>(p) + r * ld * elt_bytes<ELT>();
}
template <Elt ELT>
__device__ __forceinline__ const char* at_row(const void* p, int64_t r, int64_t ld) {
    return static_cast<const char*>(p) + r * ld * elt_bytes<ELT>();
}

// One row to a block, U units of 16 elements to a thread, eight lanes to a
// 1x128 block; the row stays in registers between its sum and its rounding.
template <Elt ELT, Elt WELT, bool RES, int U>
__global__ void __launch_bounds__(U == 1 ? 512 : 1024) norm_rows_kernel(NormArgs a, int64_t nb) {
    __shared__ float part[32];
    let_next_start();
    wait_for_stream();
    const int64_t row = blockIdx.x;
    Unit<ELT> h[U];
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t k = ((int64_t)u * blockDim.x + threadIdx.x) * 16;
        h[u].clear();
        if (k < a.K) {
            h[u].load(at_row<ELT>(a.x, row, a.ldx), k);
            if constexpr (RES) {
                Unit<ELT> r;
                r.load(at_row<ELT>(a.residual, row, a.ldr), k);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[u].set2(j, fadd(h[u].f(2 * j), r.f(2 * j)), fadd(h[u].f(2 * j + 1), r.f(2 * j + 1)));
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) sum = ffma(h[u].f(j), h[u].f(j), sum);
    }
    Unit<WELT> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t k = ((int64_t)u * blockDim.x + threadIdx.x) * 16;
        w[u].clear();
        if (k < a.K) w[u].load_shared(a.weight, k);
    }
    sum = block_sum(sum, part);
    const float rstd = rstd_of(sum, a.K, a.eps);
    if (a.rstd && threadIdx.x == 0) store_f32<Elt::FP32>(a.rstd, row, rstd);
    const bool strange = !(sum <= 3.4028235e38f);  // a NaN or an infinity in the row, or squares that overflow
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = (int64_t)u * blockDim.x + threadIdx.x, k = i * 16;
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = fmul(fmul(h[u].f(j), rstd), w[u].f(j));
        uint32_t amax = amax16(y);
        if constexpr (RES) {
            if (strange) h[u].canonical();
            if (a.h && k < a.K) h[u].store(at_row<ELT>(a.h, row, a.ldh), k);
        }
        if (a.y && k < a.K) {
            Unit<ELT> o;
#pragma unroll
            for (int j = 0; j < 8; ++j) o.set2(j, y[2 * j], y[2 * j + 1]);
            if (amax > 0x7F800000u) o.canonical();
            o.store(at_row<ELT>(a.y, row, a.K), k);
        }
        if (a.data) {
#pragma unroll
            for (int d = 1; d < 8; d *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
            const uint32_t code = scale_code128(amax);
            if (k < a.K) {
                if ((threadIdx.x & 7) == 0) a.scales[row * nb + i / 8] = (uint8_t)code;
                e4m3_store16(a.data + row * a.K + k, y, code);
            }
        }
    }
}

constexpr int kAnyThreads = 256, kAnyWarps = kAnyThreads / 32, kHeld = 8;

// Any alignment and any K: one row to a block, 1x128 blocks to its warps in
// turn, neighbours to neighbouring lanes.  The first kHeld blocks of a warp
// (rows of 8192) stay in registers, what is behind them is read again.
template <Elt ELT, bool RES>
__global__ void __launch_bounds__(kAnyThreads) norm_any_kernel(NormArgs a, int64_t nb, bool w_bf16) {
    __shared__ float part[32];
    let_next_start();
    wait_for_stream();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const void* x = at_row<ELT>(a.x, row, a.ldx);
    const void* res = RES ? at_row<ELT>(a.residual, row, a.ldr) : nullptr;
    void* hp = RES && a.h ? at_row<ELT>(a.h, row, a.ldh) : nullptr;
    const auto sum_at = [&](int64_t k) {
        float v = __uint_as_float(load_f32<ELT>(x, k));
        if constexpr (RES) {
            v = fadd(v, __uint_as_float(load_f32<ELT>(res, k)));
            if constexpr (ELT == Elt::BF16) v = __uint_as_float(bf16x2_from_f32(v, 0.0f) & 0xFFFF0000u);
        }
        return v;
    };
    float held[kHeld][4];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = ((int64_t)i * kAnyWarps + warp) * 128 + lane + 32 * q;
            held[i][q] = k < a.K ? sum_at(k) : 0.0f;
        }
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = ((int64_t)i * kAnyWarps + warp) * 128 + lane + 32 * q;
            if (hp && k < a.K) store_f32<ELT>(hp, k, held[i][q]);
            sum = ffma(held[i][q], held[i][q], sum);
        }
    for (int64_t b = kHeld * kAnyWarps + warp; b < nb; b += kAnyWarps)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = b * 128 + lane + 32 * q;
            const float v = k < a.K ? sum_at(k) : 0.0f;
            if (hp && k < a.K) store_f32<ELT>(hp, k, v);
            sum = ffma(v, v, sum);
        }
    const float rstd = rstd_of(block_sum(sum, part), a.K, a.eps);
    if (a.rstd && threadIdx.x == 0) store_f32<Elt::FP32>(a.rstd, row, rstd);
    const auto finish = [&](int64_t b, const float (&v)[4]) {
        float y[4];
        uint32_t amax = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = b * 128 + lane + 32 * q;
            const float w = k >= a.K ? 0.0f
                                     : __uint_as_float(w_bf16 ? load_f32<Elt::BF16>(a.weight, k) : load_f32<Elt::FP32>(a.weight, k));
            y[q] = k < a.K ? fmul(fmul(v[q], rstd), w) : 0.0f;
            amax = max(amax, __float_as_uint(y[q]) & 0x7FFFFFFFu);
            if (a.y && k < a.K) store_f32<ELT>(at_row<ELT>(a.y, row, a.K), k, y[q]);
        }
        if (!a.data) return;
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        const uint32_t code = scale_code128(amax);
        if (lane == 0) a.scales[row * nb + b] = (uint8_t)code;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = b * 128 + lane + 32 * q;
            if (k < a.K) a.data[row * a.K + k] = e4m3_byte(y[q], code);
        }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if ((int64_t)i * kAnyWarps + warp < nb) finish((int64_t)i * kAnyWarps + warp, held[i]);
    for (int64_t b = kHeld * kAnyWarps + warp; b < nb; b += kAnyWarps) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t k = b * 128 + lane + 32 * q;
            // h may lie over x or the residual: what this thread wrote there is read back
            v[q] = k >= a.K ? 0.0f : hp ? __uint_as_float(load_f32<ELT>(hp, k)) : sum_at(k);
        }
        finish(b, v);
    }
}

// --------------------------------------------------------------- gradient
//
// With n = h r and g the gradient of y:
//   c = mean_k(g_k w_k n_k)   d_h = r (g w - n c) + g_h   d_w = sum over rows of g n
// d_w is summed by each block over its rows, and the blocks' sums in a fixed
// order by a second kernel: no atomics.

// Rows of units: a block takes every gridDim.x-th row and keeps its columns'
// part of d_w in registers.
template <Elt ELT, Elt WELT, int U>
__global__ void __launch_bounds__(U == 1 ? 512 : 1024) norm_grad_rows_kernel(NormGradArgs a, float* parts) {
    __shared__ float part[2][32];
    let_next_start();
    wait_for_stream();
    Unit<WELT> w[U];
    float dw[U][16] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t k = ((int64_t)u * blockDim.x + threadIdx.x) * 16;
        w[u].clear();
        if (k < a.K) w[u].load_shared(a.weight, k);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        Unit<ELT> g[U], h[U];
        const float r = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = ((int64_t)u * blockDim.x + threadIdx.x) * 16;
            g[u].clear(), h[u].clear();
            if (k < a.K) {
                g[u].load(at_row<ELT>(a.g, row, a.ldg), k);
                h[u].load(at_row<ELT>(a.h, row, a.ldh), k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float n = fmul(h[u].f(j), r);
                dot = ffma(fmul(g[u].f(j), w[u].f(j)), n, dot);
                dw[u][j] = ffma(g[u].f(j), n, dw[u][j]);
            }
        const float c = fdiv(block_sum(dot, part[turn]), (float)a.K);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = ((int64_t)u * blockDim.x + threadIdx.x) * 16;
            if (k >= a.K) continue;
            Unit<ELT> o, add;
            add.clear();
            if (a.g_h) add.load(at_row<ELT>(a.g_h, row, a.ldgh), k);
            const auto value = [&](int j) {
                const float d = ffma(fmul(h[u].f(j), r), -c, fmul(g[u].f(j), w[u].f(j)));
                return ffma(d, r, add.f(j));
            };
#pragma unroll
            for (int j = 0; j < 8; ++j) o.set2(j, value(2 * j), value(2 * j + 1));
            if (!(fabsf(c) <= 3.4028235e38f)) o.canonical();
            o.store(at_row<ELT>(a.d_h, row, a.ldd), k);
        }
    }
    if (!parts) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t k = ((int64_t)u * blockDim.x + threadIdx.x) * 16;
        if (k >= a.K) continue;
        float4* p = reinterpret_cast<float4*>(parts + blockIdx.x * a.K + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = make_float4(dw[u][4 * j], dw[u][4 * j + 1], dw[u][4 * j + 2], dw[u][4 * j + 3]);
    }
}

template <Elt ELT>
__device__ __forceinline__ float weight_at(const void* w, int64_t k, bool bf16) {
    return __uint_as_float(bf16 ? load_f32<Elt::BF16>(w, k) : load_f32<Elt::FP32>(w, k));
}

// Any alignment and any K: d_h, one row to a block, read twice ...
template <Elt ELT>
__global__ void __launch_bounds__(kAnyThreads) norm_grad_any_kernel(NormGradArgs a, bool w_bf16) {
    __shared__ float part[32];
    let_next_start();
    wait_for_stream();
    const int64_t row = blockIdx.x;
    const void* g = at_row<ELT>(a.g, row, a.ldg);
    const void* h = at_row<ELT>(a.h, row, a.ldh);
    const float r = a.rstd[row];
    float dot = 0.0f;
#pragma unroll 4
    for (int64_t k = threadIdx.x; k < a.K; k += kAnyThreads)
        dot = ffma(fmul(__uint_as_float(load_f32<ELT>(g, k)), weight_at<ELT>(a.weight, k, w_bf16)),
                   fmul(__uint_as_float(load_f32<ELT>(h, k)), r), dot);
    const float c = fdiv(block_sum(dot, part), (float)a.K);
#pragma unroll 4
    for (int64_t k = threadIdx.x; k < a.K; k += kAnyThreads) {
        const float gw = fmul(__uint_as_float(load_f32<ELT>(g, k)), weight_at<ELT>(a.weight, k, w_bf16));
        const float d = ffma(fmul(__uint_as_float(load_f32<ELT>(h, k)), r), -c, gw);
        const float add = a.g_h ? __uint_as_float(load_f32<ELT>(at_row<ELT>(a.g_h, row, a.ldgh), k)) : 0.0f;
        store_f32<ELT>(at_row<ELT>(a.d_h, row, a.ldd), k, ffma(d, r, add));
    }
}

// ... and d_w, a column to a thread, every gridDim.y-th row to a block.
template <Elt ELT>
__global__ void __launch_bounds__(kAnyThreads) norm_weight_any_kernel(NormGradArgs a, float* parts) {
    let_next_start();
    wait_for_stream();
    const int64_t k = (int64_t)blockIdx.x * kAnyThreads + threadIdx.x;
    if (k >= a.K) return;
    float dw = 0.0f;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
        dw = ffma(__uint_as_float(load_f32<ELT>(at_row<ELT>(a.g, row, a.ldg), k)),
                  fmul(__uint_as_float(load_f32<ELT>(at_row<ELT>(a.h, row, a.ldh), k)), a.rstd[row]), dw);
    parts[blockIdx.y * a.K + k] = dw;
}

// d_w[k] = the blocks' sums in their order: 32 columns to a block, each of its
// eight warps an eighth of the blocks.
__global__ void __launch_bounds__(256) norm_weight_sum_kernel(const float* parts, int n, int64_t K, float* out) {
    __shared__ float part[8][32];
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t k = (int64_t)blockIdx.x * 32 + lane;
    const int per = (n + 7) / 8, end = min(n, (warp + 1) * per);
    float sum = 0.0f;
    if (k < K)
#pragma unroll 8
        for (int i = warp * per; i < end; ++i) sum = fadd(sum, parts[i * K + k]);
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && k < K) {
#pragma unroll
        for (int w = 1; w < 8; ++w) sum = fadd(sum, part[w][lane]);
        store_f32<Elt::FP32>(out, k, sum);
    }
}

unsigned unit_threads(int64_t K, int U) { return (unsigned)(ceil_div(ceil_div(K, 16 * U), 32) * 32); }

template <Elt ELT, Elt WELT, bool RES>
cudaError_t rows_launch(const NormArgs& a, cudaStream_t s) {
    const int64_t nb = ceil_div(a.K, 128);
    const dim3 grid((unsigned)a.rows);
    // 512 units of 16 to a block: a row of up to 8192 elements one a thread, up to 32768 two
    if (a.K <= 8192) return launch_overlapped(norm_rows_kernel<ELT, WELT, RES, 1>, grid, unit_threads(a.K, 1), 0, 0, s, a, nb);
    return launch_overlapped(norm_rows_kernel<ELT, WELT, RES, 2>, grid, unit_threads(a.K, 2), 0, 0, s, a, nb);
}

template <Elt ELT, bool RES>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    // rows of units: 32-byte loads and stores, 16-byte stores of payloads
    const bool units = a.K % 16 == 0 && a.K <= 32768 && unit_rows<ELT>(a.x, a.rows, a.ldx) && on_bytes(a.weight, 16) &&
                       (!RES || (unit_rows<ELT>(a.residual, a.rows, a.ldr) && unit_rows<ELT>(a.h, a.rows, a.ldh))) &&
                       unit_rows<ELT>(a.y, a.rows, a.K) && on_bytes(a.data, 16);
    if (!units)
        return launch_overlapped(norm_any_kernel<ELT, RES>, dim3((unsigned)a.rows), kAnyThreads, 0, 0, s, a, ceil_div(a.K, 128),
                                 a.weight_elt == Elt::BF16);
    return a.weight_elt == Elt::BF16 ? rows_launch<ELT, Elt::BF16, RES>(a, s) : rows_launch<ELT, Elt::FP32, RES>(a, s);
}

template <Elt ELT, Elt WELT>
cudaError_t grad_rows_launch(const NormGradArgs& a, unsigned blocks, cudaStream_t s) {
    if (a.K <= 8192)
        return launch_overlapped(norm_grad_rows_kernel<ELT, WELT, 1>, dim3(blocks), unit_threads(a.K, 1), 0, 0, s, a, a.parts);
    return launch_overlapped(norm_grad_rows_kernel<ELT, WELT, 2>, dim3(blocks), unit_threads(a.K, 2), 0, 0, s, a, a.parts);
}

template <Elt ELT>
cudaError_t grad_launch(const NormGradArgs& a, cudaStream_t s) {
    const bool units = a.K % 16 == 0 && a.K <= 16384 && unit_rows<ELT>(a.g, a.rows, a.ldg) && unit_rows<ELT>(a.h, a.rows, a.ldh) &&
                       unit_rows<ELT>(a.g_h, a.rows, a.ldgh) && unit_rows<ELT>(a.d_h, a.rows, a.ldd) && on_bytes(a.weight, 16);
    const unsigned blocks = (unsigned)(a.rows < kNormParts ? a.rows : kNormParts);
    cudaError_t e;
    if (units) {
        e = a.weight_elt == Elt::BF16 ? grad_rows_launch<ELT, Elt::BF16>(a, blocks, s) : grad_rows_launch<ELT, Elt::FP32>(a, blocks, s);
    } else {
        e = cudaSuccess;
        if (a.parts)  // ahead of d_h, which may lie over g
            e = launch_overlapped(norm_weight_any_kernel<ELT>, dim3((unsigned)ceil_div(a.K, kAnyThreads), blocks), kAnyThreads, 0, 0, s, a,
                                  a.parts);
        if (e == cudaSuccess)
            e = launch_overlapped(norm_grad_any_kernel<ELT>, dim3((unsigned)a.rows), kAnyThreads, 0, 0, s, a, a.weight_elt == Elt::BF16);
    }
    if (e == cudaSuccess && a.parts)
        e = launch_overlapped(norm_weight_sum_kernel, dim3((unsigned)ceil_div(a.K, 32)), 256, 0, 0, s, a.parts, (int)blocks, a.K, a.d_weight);
    return e;
}

}  // namespace

cudaError_t launch_norm(Elt elt, const NormArgs& a, cudaStream_t s) {
    const cudaError_t e = elt == Elt::BF16 ? (a.residual ? launch<Elt::BF16, true>(a, s) : launch<Elt::BF16, false>(a, s))
                                           : (a.residual ? launch<Elt::FP32, true>(a, s) : launch<Elt::FP32, false>(a, s));
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

cudaError_t launch_norm_grad(Elt elt, const NormGradArgs& a, cudaStream_t s) {
    const cudaError_t e = elt == Elt::BF16 ? grad_launch<Elt::BF16>(a, s) : grad_launch<Elt::FP32>(a, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace mxq
