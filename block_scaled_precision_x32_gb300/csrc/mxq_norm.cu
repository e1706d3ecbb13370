// mxq_norm.cu -- root-mean-square norm of x plus a residual, written as the
// E4M3 operand of the next product (1x128 scales), and its gradient.
//
//   h = RN(x + residual)   r = 1 / sqrt(mean_k h_k^2 + eps)   y_k = (h_k r) w_k
//
// The statistics are those of h as it is stored, so that the gradient, which
// has h alone, is that of what was computed.  y is quantized before it is
// rounded to x's type.  Sums and statistics are fp32.
#include <atomic>
#include <type_traits>

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

// Sum over the `warps` warps of a row from the block's `first` on, the same in
// each of their threads: lanes, then warps, in a fixed order.  `part` is written
// by this call alone until the block's next barrier, which every thread meets.
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float (&part)[WARPS], int first, int warps) {
    v = warp_sum(v);
    if (threadIdx.x < WARPS && threadIdx.x >= blockDim.x / 32) part[threadIdx.x] = 0.0f;  // of no warp
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    if (warps == 1) return v;
    float sum = 0.0f;
    if (warps > WARPS / 2 || warps == (int)blockDim.x / 32) {  // the row is the block's only one
#pragma unroll
        for (int w = 0; w < WARPS; w += 4) {
            const float4 q = *reinterpret_cast<const float4*>(part + w);
            sum = fadd(sum, fadd(fadd(q.x, q.y), fadd(q.z, q.w)));
        }
    } else {
#pragma unroll 4
        for (int w = first; w < first + warps; ++w) sum = fadd(sum, part[w]);
    }
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

// U units of 16 elements to a thread, eight lanes to a 1x128 block; the row
// stays in registers between its sum and its rounding.  row_threads threads to
// a row, so that short rows share a block.  8192 x 7184 bf16 with residual and y
// 77 us, 6.85 TB/s.
template <Elt ELT, Elt WELT, bool RES, int U, bool SHARED>
__global__ void __launch_bounds__(U == 1 ? 512 : 1024, U == 1 && ELT == Elt::BF16 ? 3 : 1) norm_rows_kernel(NormArgs a, int64_t nb, int threads) {
    __shared__ __align__(16) float part[U == 1 ? 16 : 32];
    let_next_start();
    wait_for_stream();
    const int row_threads = SHARED ? threads : blockDim.x, mine = SHARED ? threadIdx.x / row_threads : 0, tid = threadIdx.x - mine * row_threads;
    const int64_t row = SHARED ? (int64_t)blockIdx.x * (blockDim.x / row_threads) + mine : blockIdx.x;
    const bool real = !SHARED || row < a.rows;
    Unit<ELT> h[U];
    float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t k = ((int64_t)u * row_threads + tid) * 16;
        h[u].clear();
        if (real && k < a.K) {
            h[u].load(at_row<ELT>(a.x, row, a.ldx), k);
            if constexpr (RES) {
                Unit<ELT> r;
                r.load(at_row<ELT>(a.residual, row, a.ldr), k);
                h[u].add(r);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) squares = fma2(h[u].f2(j), h[u].f2(j), squares);
    }
    Unit<WELT> w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t k = ((int64_t)u * row_threads + tid) * 16;
        w[u].clear();
        if (k < a.K) w[u].load_shared(a.weight, k);
    }
    const float sum = row_sum(fadd(squares.x, squares.y), part, mine * (row_threads / 32), row_threads / 32);
    if (!real) return;  // whole warps
    const float rstd = rstd_of(sum, a.K, a.eps);
    if (a.rstd && tid == 0) store_f32<Elt::FP32>(a.rstd, row, rstd);
    const bool strange = !(sum <= 3.4028235e38f);  // a NaN or an infinity in the row, or squares that overflow
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = (int64_t)u * row_threads + tid, k = i * 16;
        if constexpr (RES) {
            if (strange) h[u].canonical();
            if (a.h && k < a.K) h[u].store(at_row<ELT>(a.h, row, a.ldh), k);
        }
        float y[16], top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = mul2(mul2(h[u].f2(j), both(rstd)), w[u].f2(j));
            y[2 * j] = v.x, y[2 * j + 1] = v.y;
            top = absmax3(top, v.x, v.y);
        }
        uint32_t amax = __float_as_uint(top) & 0x7FFFFFFFu;
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
                if ((tid & 7) == 0) a.scales[row * nb + i / 8] = (uint8_t)code;
                e4m3_store16(a.data + row * a.K + k, y, code);
            }
        }
    }
}

constexpr int kAnyThreads = 256, kAnyWarps = kAnyThreads / 32, kHeld = 8, kAhead = 2;

template <Elt ELT>
__device__ __forceinline__ float value_at(const void* p, int64_t k) {
    return __uint_as_float(load_f32<ELT>(p, k));
}

// Any alignment and any K: one row to a block, 1x128 blocks to its warps in
// turn, neighbours to neighbouring lanes: an element at a time, so that
// instructions bound it.  The first kHeld blocks of a warp (rows of 8192) stay
// in registers, what is behind them is read again.  Only the row's last block,
// where it is not a whole one, looks at each element's place.  Four blocks to a
// multiprocessor hide each other's barrier: 4095 x 7183 fp32 take 35.9 us, 8191 x
// 7183 bf16 with residual and y 108, with two thirds of the issue slots taken
// (three or five blocks, or blocks of 512 threads, 38 to 42 and 119 to 152;
// persistent blocks with their next rows on the way into shared memory 45 and 150:
// two of them have room, and wait at their barriers together).
template <Elt ELT, Elt WELT, bool RES>
__global__ void __launch_bounds__(kAnyThreads, 4) norm_any_kernel(NormArgs a, int nb) {
    __shared__ __align__(16) float part[kAnyWarps];
    let_next_start();
    wait_for_stream();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, K = (int)a.K;
    const void* x = at_row<ELT>(a.x, row, a.ldx);
    const void* res = RES ? at_row<ELT>(a.residual, row, a.ldr) : nullptr;
    void* hp = RES && a.h ? at_row<ELT>(a.h, row, a.ldh) : nullptr;
    void* yp = a.y ? at_row<ELT>(a.y, row, a.K) : nullptr;
    uint8_t* data = a.data ? a.data + row * a.K : nullptr;
    constexpr std::true_type kWhole{};
    constexpr std::false_type kPart{};
    const int whole_blocks = K / 128;
    // the lane's four elements of block b; zeros where it is not `there`, and behind the row
    const auto read = [&](auto whole, int b, bool there, float (&v)[4]) {
        const int k = b * 128 + lane;
        const auto at = [&](int q) { return there && (decltype(whole)::value || k + 32 * q < K); };
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = at(q) ? value_at<ELT>(x, k + 32 * q) : 0.0f;
        if constexpr (RES) {
            float r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) r[q] = at(q) ? value_at<ELT>(res, k + 32 * q) : 0.0f;
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                v[q] = fadd(v[q], r[q]), v[q + 1] = fadd(v[q + 1], r[q + 1]);
                if constexpr (ELT == Elt::BF16) {
                    const uint32_t two = bf16x2_from_f32(v[q + 1], v[q]);
                    v[q] = __uint_as_float(two << 16), v[q + 1] = __uint_as_float(two & 0xFFFF0000u);
                }
            }
        }
    };
    const auto keep = [&](auto whole, int b, const float (&v)[4], float sum) {
        const int k = b * 128 + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (hp && (decltype(whole)::value || k + 32 * q < K)) store_f32<ELT>(hp, k + 32 * q, v[q]);
            sum = ffma(v[q], v[q], sum);
        }
        return sum;
    };
    const bool tail = whole_blocks < nb && whole_blocks % kAnyWarps == warp;  // of this warp
    float held[kHeld][4], end[4], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) read(kWhole, i * kAnyWarps + warp, i * kAnyWarps + warp < whole_blocks, held[i]);
    read(kPart, whole_blocks, tail, end);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (i * kAnyWarps + warp < whole_blocks) sum = keep(kWhole, i * kAnyWarps + warp, held[i], sum);
    for (int b = kHeld * kAnyWarps + warp; b < whole_blocks; b += kAnyWarps) {
        float v[4];
        read(kWhole, b, true, v);
        sum = keep(kWhole, b, v, sum);
    }
    if (tail) sum = keep(kPart, whole_blocks, end, sum);
    // weights of the lane's four elements of block b, if it is `there`; zeros behind the row
    const auto weights = [&](auto whole, int b, bool there, float (&w)[4]) {
        const int k = b * 128 + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = 0.0f;
            if (there && (decltype(whole)::value || k + 32 * q < K)) {
                if constexpr (WELT == Elt::BF16) w[q] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.weight) + k + 32 * q) << 16);
                else w[q] = __ldg(static_cast<const float*>(a.weight) + k + 32 * q);
            }
        }
    };
    // the weights of kAhead blocks are on their way at once, the first ones while the row is summed
    float w[kAhead][4];
    const auto ahead = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) weights(kWhole, (i0 + i) * kAnyWarps + warp, (i0 + i) * kAnyWarps + warp < whole_blocks, w[i]);
    };
    ahead(0);
    const float rstd = rstd_of(row_sum(sum, part, 0, kAnyWarps), a.K, a.eps);
    if (a.rstd && threadIdx.x == 0) store_f32<Elt::FP32>(a.rstd, row, rstd);
    const auto finish = [&](auto whole, int b, const float (&v)[4], const float (&w)[4]) {
        const int k = b * 128 + lane;
        const auto at = [&](int q) { return decltype(whole)::value || k + 32 * q < K; };
        float2 y[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            y[q] = mul2(mul2(make_float2(v[2 * q], v[2 * q + 1]), both(rstd)), make_float2(w[2 * q], w[2 * q + 1]));
            if (!at(2 * q)) y[q].x = 0.0f;
            if (!at(2 * q + 1)) y[q].y = 0.0f;
        }
        const float top = absmax3(absmax3(0.0f, y[0].x, y[0].y), y[1].x, y[1].y);
        if (yp)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float f = q & 1 ? y[q / 2].y : y[q / 2].x;
                if (at(q)) store_f32<ELT>(yp, k + 32 * q, f);
            }
        if (!data) return;
        const uint32_t code = scale_code128(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top) & 0x7FFFFFFFu));
        if (lane == 0) a.scales[row * nb + b] = (uint8_t)code;
        const float2 inv = both(__uint_as_float(inv_scale128(code)));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float2 p = mul2(y[q], inv);
            const uint32_t two = code == 255u ? 0x7F7Fu : e4m3x2_from_f32(__float_as_uint(p.y), __float_as_uint(p.x));
            if (at(2 * q)) data[k + 64 * q] = (uint8_t)two;
            if (at(2 * q + 1)) data[k + 64 * q + 32] = (uint8_t)(two >> 8);
        }
    };
#pragma unroll
    for (int i0 = 0; i0 < kHeld; i0 += kAhead) {
        if (i0) ahead(i0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if ((i0 + i) * kAnyWarps + warp < whole_blocks) finish(kWhole, (i0 + i) * kAnyWarps + warp, held[i0 + i], w[i]);
    }
    for (int b = kHeld * kAnyWarps + warp; b < whole_blocks; b += kAnyWarps) {
        float v[4], w[4];
        weights(kWhole, b, true, w);
        // h may lie over x or the residual: what this thread wrote there is read back
        if (hp) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = value_at<ELT>(hp, b * 128 + lane + 32 * q);
        } else {
            read(kWhole, b, true, v);
        }
        finish(kWhole, b, v, w);
    }
    if (tail) {
        float w[4];
        weights(kPart, whole_blocks, true, w);
        finish(kPart, whole_blocks, end, w);
    }
}

// --------------------------------------------------------------- gradient
//
// With n = h r and g the gradient of y:
//   c = mean_k(g_k w_k n_k)   d_h = r (g w - n c) + g_h   d_w = sum over rows of g n
// d_w is summed by each block over its rows, and the blocks' sums in a fixed
// order by a second kernel: no atomics.

// Rows on 16 bytes: one persistent block to a multiprocessor, row_threads
// threads to a row and as many rows at a time as it has threads for.  A thread
// has P pieces of 16 bytes of a row, row_threads pieces apart.  Its part of the
// rows that come next is on its way into its own slots of shared memory
// (cp.async) while it works on one: only that keeps enough bytes in flight, as
// a block has to wait for a row's sum between reading and writing it.  The
// columns' part of d_w stays in registers.  8191 x 7184 bf16 with g_h take 78 us
// with the second kernel, 6.0 TB/s (with the loads into registers, two blocks a
// multiprocessor, 144).
constexpr int kRingBytes = 220 * 1024, kRingMost = 8;

template <int N>
__device__ __forceinline__ void copies_but(int left) {
    if constexpr (N == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == N) asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    else copies_but<N - 1>(left);
}

// Values 2j and 2j + 1 of pieces.
template <Elt ELT>
__device__ __forceinline__ float2 pair_of(const uint32_t* w, int j) {
    if constexpr (ELT == Elt::BF16) return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
}

template <Elt ELT, Elt WELT, int P>
__global__ void __launch_bounds__(512) norm_grad_rows_kernel(NormGradArgs a, int row_threads, int stages) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float part[2][16];
    let_next_start();
    wait_for_stream();
    constexpr int E = 16 / (int)elt_bytes<ELT>(), kPairs = P * E / 2;  // elements of a piece, pairs of them a thread
    const int operands = a.g_h ? 3 : 2, rows_at_once = blockDim.x / row_threads;
    const int tid = threadIdx.x % row_threads, mine = threadIdx.x / row_threads;
    const int64_t first = (int64_t)blockIdx.x * rows_at_once + mine, step = (int64_t)gridDim.x * rows_at_once;
    bool there[P];
#pragma unroll
    for (int p = 0; p < P; ++p) there[p] = ((int64_t)p * row_threads + tid) * E < a.K;
    // piece p of operand o of this thread in stage s lies at ((s * operands + o) * P + p) * blockDim.x * 16 + threadIdx.x * 16
    const uint32_t slots = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    const char* from[3] = {at_row<ELT>(a.g, first, a.ldg) + tid * 16, at_row<ELT>(a.h, first, a.ldh) + tid * 16,
                           at_row<ELT>(a.g_h ? a.g_h : a.g, first, a.ldgh) + tid * 16};
    const int64_t stride[3] = {step * a.ldg * elt_bytes<ELT>(), step * a.ldh * elt_bytes<ELT>(), step * a.ldgh * elt_bytes<ELT>()};
    int64_t next = first;
    const auto fetch = [&](int stage) {  // row `next`
        if (next < a.rows) {
            uint32_t to = slots + (uint32_t)(stage * operands * P) * blockDim.x * 16;
#pragma unroll
            for (int o = 0; o < 3; ++o) {
                if (o >= operands) break;
#pragma unroll
                for (int p = 0; p < P; ++p, to += blockDim.x * 16)
                    if (there[p]) copy16(to, from[o] + p * row_threads * 16);
                from[o] += stride[o];
            }
        }
        next += step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto read = [&](uint32_t (&v)[4 * P], int stage, int o) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint4 w = *reinterpret_cast<const uint4*>(ring + ((size_t)((stage * operands + o) * P + p) * blockDim.x + threadIdx.x) * 16);
            v[4 * p] = w.x, v[4 * p + 1] = w.y, v[4 * p + 2] = w.z, v[4 * p + 3] = w.w;
        }
    };
    for (int s = 0; s < stages; ++s) fetch(s);
    if (threadIdx.x < 16 && threadIdx.x >= blockDim.x / 32) part[0][threadIdx.x] = part[1][threadIdx.x] = 0.0f;  // of no warp
    constexpr int kWeightWords = P * E * (int)elt_bytes<WELT>() / 4;
    uint32_t w[kWeightWords];
    float2 dw[kPairs] = {};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        constexpr int N = kWeightWords / P;  // words of a piece's weights: 2, 4 or 8
        const uint2* from_w = reinterpret_cast<const uint2*>(static_cast<const char*>(a.weight) + ((int64_t)p * row_threads + tid) * E * elt_bytes<WELT>());
#pragma unroll
        for (int q = 0; q < N; q += 2) {
            const uint2 v = there[p] ? __ldg(from_w + q / 2) : make_uint2(0u, 0u);
            w[p * N + q] = v.x, w[p * N + q + 1] = v.y;
        }
    }
    const float per_k = fdiv(1.0f, (float)a.K);
    const int64_t turns = (a.rows + step - 1) / step;  // the same for every thread: each one meets every barrier
    int stage = 0;
    float next_r = first < a.rows ? a.rstd[first] : 0.0f;
    for (int64_t turn = 0; turn < turns; ++turn) {
        const int64_t row = first + turn * step;
        const float r = next_r;
        next_r = row + step < a.rows ? a.rstd[row + step] : 0.0f;
        copies_but<kRingMost - 1>(stages - 1);
        uint32_t g[4 * P], h[4 * P], add[4 * P];
        read(g, stage, 0);
        read(h, stage, 1);
        if (a.g_h) read(add, stage, 2);
#pragma unroll
        for (int i = 0; i < 4 * P; ++i) {
            if (!there[i / 4] || row >= a.rows) g[i] = h[i] = 0;
            if (!a.g_h) add[i] = 0;
        }
        float2 dot2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            dot2 = fma2(mul2(pair_of<ELT>(g, j), pair_of<WELT>(w, j)), pair_of<ELT>(h, j), dot2);
            dw[j] = fma2(pair_of<ELT>(g, j), mul2(pair_of<ELT>(h, j), both(r)), dw[j]);
        }
        float dot = warp_sum(fadd(dot2.x, dot2.y));
        float* sums = part[turn & 1];
        if ((threadIdx.x & 31) == 0) sums[threadIdx.x / 32] = dot;
        __syncthreads();
        fetch(stage);  // what was here is in registers
        stage = stage + 1 < stages ? stage + 1 : 0;
        if (row_threads > 256) {
            // the row's warps; behind the block's last there are zeros
            dot = 0.0f;
#pragma unroll
            for (int v = 0; v < 16; v += 4) {
                const float4 q = *reinterpret_cast<const float4*>(sums + v);
                dot = fadd(dot, fadd(fadd(q.x, q.y), fadd(q.z, q.w)));
            }
        } else if (row_threads > 32) {
            dot = 0.0f;
#pragma unroll 4
            for (int v = mine * (row_threads / 32); v < (mine + 1) * (row_threads / 32); ++v) dot = fadd(dot, sums[v]);
        }
        if (row >= a.rows) continue;
        const float rc = -fmul(r, fmul(fmul(r, dot), per_k));  // d_h = r g w - (r h) (r c) + g_h
        float top = 0.0f;
        uint32_t o[4 * P];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const float2 d = fma2(mul2(pair_of<ELT>(g, j), pair_of<WELT>(w, j)), both(r),
                                  fma2(mul2(pair_of<ELT>(h, j), both(r)), both(rc), pair_of<ELT>(add, j)));
            if constexpr (ELT == Elt::BF16) o[j] = bf16x2_from_f32(d.y, d.x);
            else o[2 * j] = __float_as_uint(d.x), o[2 * j + 1] = __float_as_uint(d.y);
            top = absmax3(top, d.x, d.y);
        }
        if (top != top)
#pragma unroll
            for (uint32_t& v : o) v = canonical_word<ELT>(v);
        char* to = at_row<ELT>(a.d_h, row, a.ldd) + tid * 16;
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (there[p]) st16(to + p * row_threads * 16, o[4 * p], o[4 * p + 1], o[4 * p + 2], o[4 * p + 3]);
    }
    if (!a.parts) return;
    // the rows that ran side by side add up in their order
    float2* sums = reinterpret_cast<float2*>(ring);
    copies_but<0>(0);
    for (int v = 1; v < rows_at_once; ++v) {
        __syncthreads();
        if (mine == v)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sums[j * row_threads + tid] = dw[j];
        __syncthreads();
        if (mine == 0)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float2 o = sums[j * row_threads + tid];
                dw[j] = make_float2(fadd(dw[j].x, o.x), fadd(dw[j].y, o.y));
            }
    }
    if (mine != 0) return;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (!there[p]) continue;
        float4* to = reinterpret_cast<float4*>(a.parts + blockIdx.x * a.K + ((int64_t)p * row_threads + tid) * E);
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
            const float2 x = dw[p * E / 2 + 2 * q], y = dw[p * E / 2 + 2 * q + 1];
            to[q] = make_float4(x.x, x.y, y.x, y.y);
        }
    }
}

// Rows of up to 8192 elements that do not lie on 16 bytes: a persistent block
// to a multiprocessor, every 1024th element of a row to a thread, the next row's
// on their way while it works on one.  Bound by that latency: 4095 x 7183 bf16
// take 93 us, 2.5 TB/s.
constexpr int kLooseThreads = 1024, kLoose = 8;
template <Elt ELT>
__global__ void __launch_bounds__(kLooseThreads) norm_grad_loose_kernel(NormGradArgs a, bool w_bf16) {
    __shared__ __align__(16) float part[2][kLooseThreads / 32];
    let_next_start();
    wait_for_stream();
    const int K = (int)a.K;
    // what is on its way stays as it is in memory: to touch it would be to wait for it
    using Raw = typename std::conditional<ELT == Elt::BF16, uint16_t, uint32_t>::type;
    const auto f32_of = [](Raw v) { return __uint_as_float(ELT == Elt::BF16 ? (uint32_t)v << 16 : (uint32_t)v); };
    float w[kLoose], dw[kLoose] = {};
    Raw next_g[kLoose], next_h[kLoose];
#pragma unroll
    for (int i = 0; i < kLoose; ++i) {
        const int k = i * kLooseThreads + threadIdx.x;
        w[i] = k >= K ? 0.0f : w_bf16 ? value_at<Elt::BF16>(a.weight, k) : value_at<Elt::FP32>(a.weight, k);
    }
    const auto fetch = [&](int64_t row) {
        const Raw* g = reinterpret_cast<const Raw*>(at_row<ELT>(a.g, row, a.ldg));
        const Raw* h = reinterpret_cast<const Raw*>(at_row<ELT>(a.h, row, a.ldh));
#pragma unroll
        for (int i = 0; i < kLoose; ++i) {
            const int k = i * kLooseThreads + threadIdx.x;
            const bool there = row < a.rows && k < K;
            next_g[i] = there ? g[k] : (Raw)0;
            next_h[i] = there ? h[k] : (Raw)0;
        }
    };
    const float per_k = fdiv(1.0f, (float)K);
    fetch(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const float r = a.rstd[row];
        float g[kLoose], h[kLoose], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kLoose; ++i) {
            g[i] = f32_of(next_g[i]);
            h[i] = fmul(f32_of(next_h[i]), r);
            dw[i] = ffma(g[i], h[i], dw[i]);
            g[i] = fmul(g[i], w[i]);
            dot = ffma(g[i], h[i], dot);
        }
        fetch(row + gridDim.x);
        const float c = fmul(row_sum(dot, part[turn], 0, kLooseThreads / 32), per_k);
        const Raw* add = a.g_h ? reinterpret_cast<const Raw*>(at_row<ELT>(a.g_h, row, a.ldgh)) : nullptr;
        Raw more[kLoose];  // all of them ahead of the first store, which may go to the same memory
#pragma unroll
        for (int i = 0; i < kLoose; ++i) more[i] = add && i * kLooseThreads + (int)threadIdx.x < K ? add[i * kLooseThreads + threadIdx.x] : (Raw)0;
        void* to = at_row<ELT>(a.d_h, row, a.ldd);
#pragma unroll
        for (int i = 0; i < kLoose; ++i) {
            const int k = i * kLooseThreads + threadIdx.x;
            if (k < K) store_f32<ELT>(to, k, ffma(ffma(h[i], -c, g[i]), r, f32_of(more[i])));
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int i = 0; i < kLoose; ++i)
        if (i * kLooseThreads + (int)threadIdx.x < K) a.parts[blockIdx.x * a.K + i * kLooseThreads + threadIdx.x] = dw[i];
}

template <Elt ELT>
__device__ __forceinline__ float weight_at(const void* w, int64_t k, bool bf16) {
    return __uint_as_float(bf16 ? load_f32<Elt::BF16>(w, k) : load_f32<Elt::FP32>(w, k));
}

// Any alignment and any K: d_h, one row to a block, read twice ...
template <Elt ELT>
__global__ void __launch_bounds__(kAnyThreads) norm_grad_any_kernel(NormGradArgs a, bool w_bf16) {
    __shared__ __align__(16) float part[kAnyWarps];
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
    const float c = fdiv(row_sum(dot, part, 0, kAnyWarps), (float)a.K);
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
// eight warps an eighth of the blocks.  304 x 7184 take 3 us behind the first kernel.
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
    // 512 units of 16 to a block: a row of up to 8192 elements one a thread, up to 32768 two; rows of up to 2048 share blocks of 256
    const int units = a.K <= 8192 ? 1 : 2, row_threads = (int)unit_threads(a.K, units);
    const int rows = row_threads <= 128 && a.rows > sm_count() ? 256 / row_threads : 1;
    const dim3 grid((unsigned)ceil_div(a.rows, rows));
    const int64_t nb = ceil_div(a.K, 128);
    return units > 1 ? launch_overlapped(norm_rows_kernel<ELT, WELT, RES, 2, false>, grid, row_threads, 0, 0, s, a, nb, row_threads)
           : rows > 1 ? launch_overlapped(norm_rows_kernel<ELT, WELT, RES, 1, true>, grid, rows * row_threads, 0, 0, s, a, nb, row_threads)
                      : launch_overlapped(norm_rows_kernel<ELT, WELT, RES, 1, false>, grid, row_threads, 0, 0, s, a, nb, row_threads);
}

template <Elt ELT, bool RES>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
    // rows of units: 32-byte loads and stores, 16-byte stores of payloads
    const bool units = a.K % 16 == 0 && a.K <= 32768 && unit_rows<ELT>(a.x, a.rows, a.ldx) && on_bytes(a.weight, 16) &&
                       (!RES || (unit_rows<ELT>(a.residual, a.rows, a.ldr) && unit_rows<ELT>(a.h, a.rows, a.ldh))) &&
                       unit_rows<ELT>(a.y, a.rows, a.K) && on_bytes(a.data, 16);
    if (!units)
        return a.weight_elt == Elt::BF16
                   ? launch_overlapped(norm_any_kernel<ELT, Elt::BF16, RES>, dim3((unsigned)a.rows), kAnyThreads, 0, 0, s, a, (int)ceil_div(a.K, 128))
                   : launch_overlapped(norm_any_kernel<ELT, Elt::FP32, RES>, dim3((unsigned)a.rows), kAnyThreads, 0, 0, s, a, (int)ceil_div(a.K, 128));
    return a.weight_elt == Elt::BF16 ? rows_launch<ELT, Elt::BF16, RES>(a, s) : rows_launch<ELT, Elt::FP32, RES>(a, s);
}

// Stages of the ring that shared memory has room for, 0 where rows are too long for it.
struct RingShape {
    int wide, row_threads, threads, stages;
    size_t bytes;
};
template <Elt ELT>
RingShape ring_shape(const NormGradArgs& a) {
    RingShape r{};
    r.wide = a.K > 8192;  // 16 elements a thread, or 32
    r.row_threads = (int)unit_threads(a.K, r.wide ? 2 : 1);
    if (r.row_threads > 512) return r;
    r.threads = 512 / r.row_threads * r.row_threads;
    const size_t elements = (size_t)r.threads * (r.wide ? 32 : 16), stage = (a.g_h ? 3 : 2) * elements * elt_bytes<ELT>();
    r.stages = (int)(kRingBytes / stage < kRingMost ? kRingBytes / stage : kRingMost);
    if (r.stages < 2) r.stages = 0;
    const size_t sums = (size_t)r.row_threads * (r.wide ? 32 : 16) * 4;
    r.bytes = r.stages * stage > sums ? r.stages * stage : sums;
    return r;
}

template <Elt ELT, Elt WELT, int P>
cudaError_t grad_rows_launch(const NormGradArgs& a, const RingShape& r, unsigned blocks, cudaStream_t s) {
    static std::atomic<bool> allowed[kDevices];
    const cudaError_t e = allow_shared_memory(norm_grad_rows_kernel<ELT, WELT, P>, kRingBytes, allowed);
    if (e != cudaSuccess) return e;
    return launch_overlapped(norm_grad_rows_kernel<ELT, WELT, P>, dim3(blocks), r.threads, r.bytes, 0, s, a, r.row_threads, r.stages);
}
template <Elt ELT, Elt WELT>
cudaError_t grad_rows_launch(const NormGradArgs& a, const RingShape& r, unsigned blocks, cudaStream_t s) {
    constexpr int P = (int)elt_bytes<ELT>();  // pieces of 16 elements
    return r.wide ? grad_rows_launch<ELT, WELT, 2 * P>(a, r, blocks, s) : grad_rows_launch<ELT, WELT, P>(a, r, blocks, s);
}

template <Elt ELT>
cudaError_t grad_launch(const NormGradArgs& a, cudaStream_t s) {
    const auto on16 = [&](const void* p, int64_t ld) { return on_bytes(p, 16) && (a.rows <= 1 || ld * elt_bytes<ELT>() % 16 == 0); };
    const bool pieces = a.K * elt_bytes<ELT>() % 16 == 0 && a.K <= 16384 && on16(a.g, a.ldg) && on16(a.h, a.ldh) && on16(a.g_h, a.ldgh) &&
                        on16(a.d_h, a.ldd) && on_bytes(a.weight, 16);
    const RingShape ring = pieces ? ring_shape<ELT>(a) : RingShape{};
    unsigned blocks;
    cudaError_t e;
    if (ring.stages) {
        const int64_t groups = ceil_div(a.rows, ring.threads / ring.row_threads), most = sm_count() < kNormParts ? sm_count() : kNormParts;
        blocks = (unsigned)(groups < most ? groups : most);
        e = a.weight_elt == Elt::BF16 ? grad_rows_launch<ELT, Elt::BF16>(a, ring, blocks, s) : grad_rows_launch<ELT, Elt::FP32>(a, ring, blocks, s);
    } else if (a.K <= kLoose * kLooseThreads) {
        const int64_t most = sm_count() < kNormParts ? sm_count() : kNormParts;
        blocks = (unsigned)(a.rows < most ? a.rows : most);
        e = launch_overlapped(norm_grad_loose_kernel<ELT>, dim3(blocks), kLooseThreads, 0, 0, s, a, a.weight_elt == Elt::BF16);
    } else {
        blocks = (unsigned)(a.rows < kNormParts ? a.rows : kNormParts);
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
