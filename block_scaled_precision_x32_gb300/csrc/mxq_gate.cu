// mxq_gate.cu -- the gated activation between an expert's two products,
//
//   a[r, k] = silu(x[r, k]) x[r, H + k],   silu(v) = v / (1 + exp(-v)),
//
// in x's type, as the E4M3 operand of the second product (1x128 scales), or of
// its weight's gradient (128x1), and its gradient.  Arithmetic is fp32; one
// rounding at the end.
#include "mxq_device.cuh"
#include "mxq_e4m3.cuh"
#include "mxq_layer.h"
#include "mxq_launch.cuh"

namespace mxq {
namespace {

__device__ __forceinline__ float gated(float gate, float up) { return fmul(fmul(gate, Sigmoid(gate).s), up); }

// Rows of 16-element units, eight lanes to a 1x128 block.
template <Elt ELT, bool QUANT>
__global__ void __launch_bounds__(256) gate_rows_kernel(GateArgs a, int64_t nb) {
    let_next_start();
    wait_for_stream();
    const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int64_t row, b;
    split_index(unit >> 3, nb, row, b);
    const int64_t k = b * 128 + (threadIdx.x & 7) * 16;
    const bool there = row < a.rows && k < a.H;
    Unit<ELT> gate, up;
    gate.clear(), up.clear();
    if (there) {
        gate.load(a.x, row * a.ldx + k);
        up.load(a.x, row * a.ldx + a.H + k);
    }
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = gated(gate.f(j), up.f(j));
    uint32_t amax = amax16(v);
    if constexpr (QUANT) {
#pragma unroll
        for (int d = 1; d < 8; d *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        const uint32_t code = scale_code128(amax);
        if (!there) return;
        if ((threadIdx.x & 7) == 0) a.scales[row * nb + b] = (uint8_t)code;
        e4m3_store16(a.data + row * a.H + k, v, code);
    } else {
        if (!there) return;
        Unit<ELT> o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.set2(j, v[2 * j], v[2 * j + 1]);
        if (amax > 0x7F800000u) o.canonical();
        o.store(a.out, row * a.H + k);
    }
}

// Any alignment and any H: a warp per two 1x128 blocks, an element at a time,
// neighbours to neighbouring lanes.
template <Elt ELT, bool QUANT>
__global__ void __launch_bounds__(256) gate_any_kernel(GateArgs a, int64_t nb) {
    let_next_start();
    wait_for_stream();
    constexpr int B = 2;
    const int64_t first = ((int64_t)blockIdx.x * 8 + threadIdx.x / 32) * B;
    const int lane = threadIdx.x & 31;
    uint32_t gate[B][4], up[B][4];
    int64_t row[B], k0[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        split_index(first + i, nb, row[i], k0[i]);
        k0[i] = k0[i] * 128 + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool there = row[i] < a.rows && k0[i] + 32 * j < a.H;
            gate[i][j] = there ? load_f32<ELT>(a.x, row[i] * a.ldx + k0[i] + 32 * j) : 0u;
            up[i][j] = there ? load_f32<ELT>(a.x, row[i] * a.ldx + a.H + k0[i] + 32 * j) : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        if (row[i] >= a.rows) break;
        float v[4];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = gated(__uint_as_float(gate[i][j]), __uint_as_float(up[i][j]));
            amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        }
        if constexpr (QUANT) amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        const uint32_t code = scale_code128(amax);
        if (QUANT && lane == 0) a.scales[first + i] = (uint8_t)code;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k0[i] + 32 * j < a.H) {
                const int64_t at = row[i] * a.H + k0[i] + 32 * j;
                if constexpr (QUANT) a.data[at] = e4m3_byte(v[j], code);
                else store_f32<ELT>(a.out, at, v[j]);
            }
    }
}

// 128 rows x 64 columns a block, 16 rows of one column a thread, an element at
// a time: any alignment and any H.
template <Elt ELT>
__global__ void __launch_bounds__(512) gate_columns_kernel(GateArgs a) {
    let_next_start();
    wait_for_stream();
    constexpr int R = 16, Y = 8;
    __shared__ uint32_t top[Y][64];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + tx, r0 = (int64_t)blockIdx.y * 128 + ty;
    float v[R];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + Y * i;
        const bool there = r < a.rows && c < a.H;
        const uint32_t gate = there ? load_f32<ELT>(a.x, r * a.ldx + c) : 0u, up = there ? load_f32<ELT>(a.x, r * a.ldx + a.H + c) : 0u;
        v[i] = gated(__uint_as_float(gate), __uint_as_float(up));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    top[ty][tx] = amax;
    __syncthreads();
    if (c >= a.H) return;
#pragma unroll
    for (int y = 0; y < Y; ++y) amax = max(amax, top[y][tx]);
    const uint32_t code = scale_code128(amax);
    if (ty == 0) a.scales[(int64_t)blockIdx.y * a.H + c] = (uint8_t)code;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (r0 + Y * i < a.rows) a.data[(r0 + Y * i) * a.H + c] = e4m3_byte(v[i], code);
}

struct GateGrad {
    float gate, up;
    // d_up = g silu(gate);  d_gate = g up (s + silu(gate) (1 - s))
    __device__ __forceinline__ GateGrad(float g, float x, float u) {
        const Sigmoid s(x);
        const float silu = fmul(x, s.s);
        up = fmul(g, silu);
        gate = fmul(fmul(g, u), ffma(silu, s.rest, s.s));
    }
};

// A unit of 16 elements of both halves a thread.
template <Elt ELT>
__global__ void __launch_bounds__(256) gate_grad_kernel(GateArgs a, int64_t nu) {
    let_next_start();
    wait_for_stream();
    int64_t row, u;
    split_index((int64_t)blockIdx.x * 256 + threadIdx.x, nu, row, u);
    if (row >= a.rows) return;
    const int64_t k = u * 16;
    Unit<ELT> g, gate, up;
    g.load(a.g, row * a.ldg + k);
    gate.load(a.x, row * a.ldx + k);
    up.load(a.x, row * a.ldx + a.H + k);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const GateGrad p(g.f(2 * j), gate.f(2 * j), up.f(2 * j)), q(g.f(2 * j + 1), gate.f(2 * j + 1), up.f(2 * j + 1));
        gate.set2(j, p.gate, q.gate);
        up.set2(j, p.up, q.up);
        top = max(max(top, __float_as_uint(p.gate) & 0x7FFFFFFFu), __float_as_uint(q.gate) & 0x7FFFFFFFu);
        top = max(max(top, __float_as_uint(p.up) & 0x7FFFFFFFu), __float_as_uint(q.up) & 0x7FFFFFFFu);
    }
    if (top > 0x7F800000u) gate.canonical(), up.canonical();
    gate.store(a.out, row * 2 * a.H + k);
    up.store(a.out, row * 2 * a.H + a.H + k);
}

// Any alignment and any H: an element a thread.
template <Elt ELT>
__global__ void __launch_bounds__(256) gate_grad_any_kernel(GateArgs a) {
    let_next_start();
    wait_for_stream();
    int64_t row, k;
    split_index((int64_t)blockIdx.x * 256 + threadIdx.x, a.H, row, k);
    if (row >= a.rows) return;
    const GateGrad d(__uint_as_float(load_f32<ELT>(a.g, row * a.ldg + k)), __uint_as_float(load_f32<ELT>(a.x, row * a.ldx + k)),
                     __uint_as_float(load_f32<ELT>(a.x, row * a.ldx + a.H + k)));
    store_f32<ELT>(a.out, row * 2 * a.H + k, d.gate);
    store_f32<ELT>(a.out, row * 2 * a.H + a.H + k, d.up);
}

constexpr int64_t kMostBlocks = INT64_C(0x7FFFFFFF);

template <Elt ELT>
cudaError_t launch(GateForm form, const GateArgs& a, cudaStream_t s) {
    // units: rows and both halves on 32 bytes
    const bool units = a.H % 16 == 0 && unit_rows<ELT>(a.x, a.rows, a.ldx) && a.H * elt_bytes<ELT>() % 32 == 0;
    const int64_t nb = ceil_div(a.H, 128);
    if (form == GateForm::GRAD) {
        if (units && unit_rows<ELT>(a.g, a.rows, a.ldg) && on_bytes(a.out, 32)) {
            const int64_t grid = ceil_div(a.rows * (a.H / 16), 256);
            if (grid > kMostBlocks) return cudaErrorInvalidValue;
            return launch_overlapped(gate_grad_kernel<ELT>, dim3((unsigned)grid), 256, 0, 0, s, a, a.H / 16);
        }
        const int64_t grid = ceil_div(a.rows * a.H, 256);
        if (grid > kMostBlocks) return cudaErrorInvalidValue;
        return launch_overlapped(gate_grad_any_kernel<ELT>, dim3((unsigned)grid), 256, 0, 0, s, a);
    }
    if (form == GateForm::COLUMNS) {
        // blockIdx.y reaches 65535: 2^23 rows at a time
        for (int64_t r0 = 0; r0 < a.rows; r0 += INT64_C(128) * 65535) {
            GateArgs p = a;
            p.rows = a.rows - r0 < INT64_C(128) * 65535 ? a.rows - r0 : INT64_C(128) * 65535;
            p.x = static_cast<const char*>(a.x) + r0 * a.ldx * elt_bytes<ELT>();
            p.data = a.data + r0 * a.H;
            p.scales = a.scales + r0 / 128 * a.H;
            const cudaError_t e = launch_overlapped(gate_columns_kernel<ELT>,
                                                    dim3((unsigned)ceil_div(a.H, 64), (unsigned)ceil_div(p.rows, 128)), 512, 0, 0, s, p);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    const bool quant = form == GateForm::ROWS;
    if (ceil_div(a.rows * nb, 16) > kMostBlocks) return cudaErrorInvalidValue;
    if (units && (quant ? on_bytes(a.data, 16) : on_bytes(a.out, 32))) {
        const dim3 grid((unsigned)ceil_div(a.rows * nb * 8, 256));
        return quant ? launch_overlapped(gate_rows_kernel<ELT, true>, grid, 256, 0, 0, s, a, nb)
                     : launch_overlapped(gate_rows_kernel<ELT, false>, grid, 256, 0, 0, s, a, nb);
    }
    const dim3 grid((unsigned)ceil_div(a.rows * nb, 16));
    return quant ? launch_overlapped(gate_any_kernel<ELT, true>, grid, 256, 0, 0, s, a, nb)
                 : launch_overlapped(gate_any_kernel<ELT, false>, grid, 256, 0, 0, s, a, nb);
}

}  // namespace

cudaError_t launch_gate(Elt elt, GateForm form, const GateArgs& a, cudaStream_t s) {
    const cudaError_t e = elt == Elt::BF16 ? launch<Elt::BF16>(form, a, s) : launch<Elt::FP32>(form, a, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace mxq
