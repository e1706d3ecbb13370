// mxq_moe.cu -- tokens to the experts' order and back: a stable counting
// sort of the router's choices, the gather of rows, their weighted sum, and
// the gradients of both.
#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

// ------------------------------------------------------------------- sort

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kChunk = 4096;  // choices per block
constexpr int kPerWarp = kChunk / kSortWarps;

// Adds each warp's choices to its own histogram hist[warp][expert].  A warp's
// choices are consecutive and taken 32 at a time, so that a choice's rank
// among those of its expert is the count before its step plus the lanes below
// it with the same expert: the order is that of the choices.
template <typename F>
__device__ __forceinline__ void walk_choices(const MoeSortArgs& a, int64_t chunk, int* hist, F&& f) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    int* mine = hist + warp * a.experts;
    const int64_t first = chunk * kChunk + warp * kPerWarp;
    for (int i = 0; i < kPerWarp; i += 32) {
        const int64_t c = first + i + lane;
        if (first + i >= a.choices) break;
        const int id = c < a.choices ? a.ids[c] : -1;
        const bool valid = id >= 0 && id < a.experts;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, valid ? id : -1);
        const int before = valid ? mine[id] : 0;
        const int rank = __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (valid && rank == 0) mine[id] = before + __popc(same);
        __syncwarp();
        if (c < a.choices) f(c, valid, id, before + rank);
    }
}

__device__ __forceinline__ void count_chunk(const MoeSortArgs& a, int64_t chunk, int* hist) {
    for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    walk_choices(a, chunk, hist, [](int64_t, bool, int, int) {});
    __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(MoeSortArgs a) {
    extern __shared__ int hist[];
    count_chunk(a, blockIdx.x, hist);
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
        int n = 0;
        for (int w = 0; w < kSortWarps; ++w) n += hist[w * a.experts + e];
        a.counts[blockIdx.x * a.experts + e] = n;
    }
}

// Every block finds all experts' totals and where each part begins, then the
// rows of its own choices.  With one chunk the counts come from the block's
// own histogram, else from count_kernel's.
__global__ void __launch_bounds__(kSortThreads) place_kernel(MoeSortArgs a, int chunks) {
    extern __shared__ int smem[];
    const int E = (int)a.experts;
    int* hist = smem;                    // [warps][E]
    int* begin = smem + kSortWarps * E;  // [E + 1]
    int* total = begin + E + 1;          // [E]
    int* mine = total + E;               // [E]: this chunk's first rank
    count_chunk(a, blockIdx.x, hist);
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int sum = 0, before = 0;
        if (chunks == 1) {
            for (int w = 0; w < kSortWarps; ++w) sum += hist[w * E + e];
        } else {
            for (int c = 0; c < chunks; ++c) {
                if (c == (int)blockIdx.x) before = sum;
                sum += a.counts[(int64_t)c * E + e];
            }
        }
        total[e] = sum;
        mine[e] = before;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // exclusive scan of the rounded-up totals
        int64_t run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const int64_t room = e < E ? (total[e] + a.align - 1) / a.align * a.align : 0;
            int64_t incl = room;
            for (int d = 1; d < 32; d *= 2) {
                const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if ((int)threadIdx.x >= d) incl += up;
            }
            if (e < E) begin[e] = (int)(run + incl - room);
            run += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (threadIdx.x == 0) begin[E] = (int)run;
    }
    __syncthreads();
    // hist[w][e] becomes the row of the warp's first choice of e
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int row = begin[e] + mine[e];
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = hist[w * E + e];
            hist[w * E + e] = row;
            row += n;
        }
    }
    __syncthreads();
    walk_choices(a, blockIdx.x, hist, [&](int64_t c, bool valid, int, int row) {
        a.slots[c] = valid ? row : -1;
        if (valid) a.source[row] = (int)c;
    });
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += kSortThreads) a.offsets[e] = begin[e];
    // rows without a choice: behind each part, and behind the last
    for (int e = blockIdx.x; e < E; e += gridDim.x)
        for (int r = begin[e] + total[e] + threadIdx.x; r < begin[e + 1]; r += kSortThreads) a.source[r] = -1;
    for (int64_t r = begin[E] + (int64_t)blockIdx.x * kSortThreads + threadIdx.x; r < a.capacity;
         r += (int64_t)gridDim.x * kSortThreads)
        a.source[r] = -1;
}

// ------------------------------------------------------------------- rows

template <Elt ELT>
__device__ __forceinline__ float load(const void* p, int64_t i) {
    if constexpr (ELT == Elt::BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    return static_cast<const float*>(p)[i];
}

template <Elt ELT>
__device__ __forceinline__ void store(void* p, int64_t i, float v) {
    uint32_t u = __float_as_uint(v);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0x7FC00000u;
    if constexpr (ELT == Elt::BF16)
        static_cast<uint16_t*>(p)[i] = (uint16_t)bf16_rne(u);
    else
        static_cast<uint32_t*>(p)[i] = u;
}

constexpr int kRowThreads = 256;

template <Elt ELT>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(MoeRowsArgs a) {
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        const int c = a.source[r];
        const int64_t t = c < 0 ? -1 : c / a.topk;
        const bool there = t >= 0 && t < a.T;
        for (int64_t h = threadIdx.x; h < a.H; h += kRowThreads)
            if constexpr (ELT == Elt::BF16)
                static_cast<uint16_t*>(a.out)[r * a.H + h] =
                    there ? static_cast<const uint16_t*>(a.tokens)[t * a.ld_tokens + h] : (uint16_t)0;
            else
                static_cast<uint32_t*>(a.out)[r * a.H + h] =
                    there ? static_cast<const uint32_t*>(a.tokens)[t * a.ld_tokens + h] : 0u;
    }
}

template <Elt ELT>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(MoeRowsArgs a) {
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
        for (int64_t h = threadIdx.x; h < a.H; h += kRowThreads) {
            float sum = 0.0f;
            for (int64_t j = 0; j < a.topk; ++j) {
                const int64_t r = a.slots[t * a.topk + j];
                if (r < 0 || r >= a.R) continue;
                const float y = load<ELT>(a.rows, r * a.ld_rows + h);
                sum = a.weights ? fmaf(a.weights[t * a.topk + j], y, sum) : sum + y;
            }
            store<ELT>(a.out, t * a.H + h, sum);
        }
}

template <Elt ELT>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(MoeRowsArgs a) {
    __shared__ float part[kRowThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t n = a.T * a.topk;
    for (int64_t c = blockIdx.x; c < n; c += gridDim.x) {
        const int64_t t = c / a.topk, r = a.slots[c];
        const bool there = r >= 0 && r < a.R;
        float dot = 0.0f;
        if (there) {
            const float w = a.weights[c];
            for (int64_t h = threadIdx.x; h < a.H; h += kRowThreads) {
                const float g = load<ELT>(a.tokens, t * a.ld_tokens + h);
                dot = fmaf(g, load<ELT>(a.rows, r * a.ld_rows + h), dot);
                store<ELT>(a.out, r * a.H + h, w * g);
            }
        }
        for (int d = 16; d; d /= 2) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
        if (lane == 0) part[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.0f;
            for (int w = 0; w < kRowThreads / 32; ++w) sum += part[w];
            a.d_weights[c] = there ? sum : 0.0f;
        }
        __syncthreads();
    }
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        if (a.source[r] >= 0 && a.source[r] < n) continue;
        for (int64_t h = threadIdx.x; h < a.H; h += kRowThreads) store<ELT>(a.out, r * a.H + h, 0.0f);
    }
}

unsigned row_grid(int64_t rows) {
    const int64_t most = (int64_t)sm_count() * 64;
    return (unsigned)(rows < 1 ? 1 : rows < most ? rows : most);
}

}  // namespace

int64_t moe_sort_chunks(int64_t choices) { return ceil_div(choices, kChunk); }

cudaError_t launch_moe_sort(const MoeSortArgs& a, cudaStream_t s) {
    const int chunks = (int)moe_sort_chunks(a.choices);
    const int hist = (int)(kSortWarps * a.experts * 4), place = hist + (int)(3 * a.experts + 1) * 4;
    if (place > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, hist);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, place);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
    }
    if (chunks > 1) {
        count_kernel<<<chunks, kSortThreads, hist, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    place_kernel<<<chunks, kSortThreads, place, s>>>(a, chunks);
    return cudaGetLastError();
}

cudaError_t launch_moe_dispatch(Elt elt, const MoeRowsArgs& a, cudaStream_t s) {
    if (elt == Elt::BF16)
        dispatch_kernel<Elt::BF16><<<row_grid(a.R), kRowThreads, 0, s>>>(a);
    else
        dispatch_kernel<Elt::FP32><<<row_grid(a.R), kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine(Elt elt, const MoeRowsArgs& a, cudaStream_t s) {
    if (elt == Elt::BF16)
        combine_kernel<Elt::BF16><<<row_grid(a.T), kRowThreads, 0, s>>>(a);
    else
        combine_kernel<Elt::FP32><<<row_grid(a.T), kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine_grad(Elt elt, const MoeRowsArgs& a, cudaStream_t s) {
    const int64_t work = a.T * a.topk > a.R ? a.T * a.topk : a.R;
    if (elt == Elt::BF16)
        combine_grad_kernel<Elt::BF16><<<row_grid(work), kRowThreads, 0, s>>>(a);
    else
        combine_grad_kernel<Elt::FP32><<<row_grid(work), kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mxq
