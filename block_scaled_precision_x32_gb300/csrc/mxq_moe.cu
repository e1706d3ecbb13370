// mxq_moe.cu -- tokens to the experts' order and back: a stable counting
// sort of the router's choices, the gather of rows, their weighted sum, and
// the gradients of both.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mxq_device.cuh"
#include "mxq_layer.h"
#include "mxq_launch.cuh"

namespace mxq {
namespace {

// ------------------------------------------------------------------- sort

constexpr int kChunk = 4096;  // choices per block
constexpr int kHistograms = 128 * 1024;  // bytes of place_kernel's histograms, at most
constexpr int kMostExperts = 2048;       // that mxq_moe_sort takes

// Choices of the block that a walking warp takes: consecutive ones.
__device__ __forceinline__ void warp_range(const MoeSortArgs& a, int walkers, int64_t& first, int64_t& end) {
    const int warp = threadIdx.x / 32, per_warp = (kChunk / 32 + walkers - 1) / walkers * 32;
    const int64_t begin = (int64_t)blockIdx.x * kChunk;
    end = min(begin + kChunk, a.choices);
    first = min(begin + (int64_t)warp * per_warp, end);
    end = warp < walkers ? min(first + per_warp, end) : first;
}

// Histogram of the block's choices, one for each walking warp ([walkers][E])
// or one for all.
template <bool PER_WARP>
__device__ __forceinline__ void count_chunk(const MoeSortArgs& a, int walkers, int* hist) {
    const int E = (int)a.experts;
    for (int i = threadIdx.x; i < (PER_WARP ? walkers : 1) * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    int64_t first, end;
    warp_range(a, walkers, first, end);
    int* mine = hist + (PER_WARP ? threadIdx.x / 32 * E : 0);
    for (int64_t c = first + (threadIdx.x & 31); c < end; c += 32) {
        const int id = a.ids[c];
        if (id >= 0 && id < E) atomicAdd(&mine[id], 1);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(1024) count_kernel(MoeSortArgs a, int walkers) {
    extern __shared__ int hist[];
    let_next_start();
    wait_for_stream();
    count_chunk<false>(a, walkers, hist);
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[blockIdx.x * a.experts + e] = hist[e];
}

// Every block finds all experts' totals and where each part begins, then the
// rows of its own choices.  With one chunk the counts come from the block's
// own histogram, else from count_kernel's, summed by as many threads an
// expert as the block has.  Latency: 48 x 2 choices 3.5 us; 65536 x 8 over 256
// experts 14.4 us in two launches, of which the scattered stores of `source`
// and every block's sum over all chunks' counts take the most.
__global__ void __launch_bounds__(1024) place_kernel(MoeSortArgs a, int chunks, int walkers) {
    extern __shared__ int smem[];
    let_next_start();
    wait_for_stream();
    const int E = (int)a.experts;
    int* hist = smem;                 // [walkers][E]
    int* begin = smem + walkers * E;  // [E + 1]
    int* total = begin + E + 1;       // [E]
    int* mine = total + E;            // [E]: this chunk's first rank
    for (int e = threadIdx.x; e < E; e += blockDim.x) total[e] = mine[e] = 0;
    count_chunk<true>(a, walkers, hist);
    if (chunks == 1) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            int sum = 0;
            for (int w = 0; w < walkers; ++w) sum += hist[w * E + e];
            total[e] = sum;
        }
    } else {
        const int parts = max(1, (int)blockDim.x / E), step = (chunks + parts - 1) / parts;
        for (int i = threadIdx.x; i < parts * E; i += blockDim.x) {
            const int e = i % E, c0 = i / E * step, c1 = min(chunks, c0 + step);
            int sum = 0, before = 0;
#pragma unroll 16
            for (int c = c0; c < c1; ++c) {
                const int n = a.counts[(int64_t)c * E + e];
                sum += n;
                before += c < (int)blockIdx.x ? n : 0;
            }
            if (sum) atomicAdd(&total[e], sum);
            if (before) atomicAdd(&mine[e], before);
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // exclusive scan of the rounded-up totals; their sum is the capacity at most, which is an int
        const int align = (int)a.align;
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const int n = e < E ? total[e] : 0, room = align == 1 ? n : (n + align - 1) / align * align;
            int incl = room;
            for (int d = 1; d < 32; d *= 2) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if ((int)threadIdx.x >= d) incl += up;
            }
            if (e < E) begin[e] = run + incl - room;
            run += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (threadIdx.x == 0) begin[E] = run;
    }
    __syncthreads();
    // hist[w][e] becomes the row of the warp's first choice of e
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int row = begin[e] + mine[e];
        for (int w = 0; w < walkers; ++w) {
            const int n = hist[w * E + e];
            hist[w * E + e] = row;
            row += n;
        }
    }
    __syncthreads();
    // A warp takes its choices 32 at a time, so that a choice's rank among those of its expert is the count before its step
    // plus the lanes below it with the same expert: the order is that of the choices.  Lanes with the same expert are
    // found bit by bit (__match_any_sync took about five times as long here).
    int64_t first, end;
    warp_range(a, walkers, first, end);
    int* mine_w = hist + threadIdx.x / 32 * E;
    const int lane = threadIdx.x & 31, bits = 32 - __clz(E);
    for (int64_t c0 = first; c0 < end; c0 += 32) {
        const int64_t c = c0 + lane;
        int id = c < end ? a.ids[c] : -1;
        const bool valid = id >= 0 && id < E;
        id = valid ? id : E;
        unsigned same = 0xFFFFFFFFu;
        for (int b = 0; b < bits; ++b) {
            const unsigned set = __ballot_sync(0xFFFFFFFFu, id >> b & 1);
            same &= id >> b & 1 ? set : ~set;
        }
        const int row = valid ? mine_w[id] + __popc(same & ((1u << lane) - 1u)) : -1;
        __syncwarp();
        if (valid && (same >> lane) == 1u) mine_w[id] = row + 1;  // the last lane of the expert
        __syncwarp();
        if (c < end) a.slots[c] = row;
        if (valid) a.source[row] = (int)c;
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += blockDim.x) a.offsets[e] = begin[e];
    // rows without a choice: behind each part (a warp each), and behind the last
    if (a.align > 1)
        for (int e = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; e < E; e += gridDim.x * (blockDim.x / 32))
            // 64 bits: a part may end within 32 rows of 2^31
            for (int64_t r = (int64_t)begin[e] + total[e] + (threadIdx.x & 31); r < begin[e + 1]; r += 32) a.source[r] = -1;
    for (int64_t r = begin[E] + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.capacity;
         r += (int64_t)gridDim.x * blockDim.x)
        a.source[r] = -1;
}

// ------------------------------------------------------------------- rows

constexpr int kRowThreads = 256;
constexpr int kTogether = 4;  // choices of a token taken at a time

// A thread's piece of a row of H elements: VEC consecutive ones, 16 or 32
// bytes, or, where rows do not begin on 32 bytes (VEC 0), up to eight that
// lie a block's threads apart, so that lanes still touch neighbours.
template <Elt ELT, int VEC, int THREADS>
struct Piece {
    static constexpr int kBytes = ELT == Elt::BF16 ? 2 : 4;
    static constexpr int kWords = VEC ? VEC * kBytes / 4 : 8;
    static constexpr int kValues = VEC ? VEC : 8;
    uint32_t w[kWords];

    // Pieces of a row, and the first element of piece i (VEC 0: a multiple of
    // THREADS pieces, the last ones reach behind the row).
    static __device__ __forceinline__ int64_t count(int64_t H) {
        return VEC ? H / (VEC ? VEC : 1) : (H + 8 * THREADS - 1) / (8 * THREADS) * THREADS;
    }
    static __device__ __forceinline__ int64_t first(int64_t i) {
        return VEC ? i * VEC : i / THREADS * (8 * THREADS) + i % THREADS;
    }
    __device__ __forceinline__ void read(const void* row, int64_t i, int64_t H) {
        const char* p = static_cast<const char*>(row) + first(i) * kBytes;
        if constexpr (VEC == 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                w[q] = 0;
                if (first(i) + q * THREADS < H) {
                    if constexpr (ELT == Elt::BF16)
                        w[q] = reinterpret_cast<const uint16_t*>(p)[q * THREADS];
                    else
                        w[q] = reinterpret_cast<const uint32_t*>(p)[q * THREADS];
                }
            }
        } else if constexpr (kWords == 4) {
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "l"(p));
        } else {
            ld32(w, p);
        }
    }
    __device__ __forceinline__ void write(void* row, int64_t i, int64_t H) const {
        char* p = static_cast<char*>(row) + first(i) * kBytes;
        if constexpr (VEC == 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (first(i) + q * THREADS < H) {
                    if constexpr (ELT == Elt::BF16)
                        reinterpret_cast<uint16_t*>(p)[q * THREADS] = (uint16_t)w[q];
                    else
                        reinterpret_cast<uint32_t*>(p)[q * THREADS] = w[q];
                }
        } else if constexpr (kWords == 4) {
            st16(p, w[0], w[1], w[2], w[3]);
        } else {
            st32(p, w);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& v : w) v = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (ELT == Elt::FP32) return __uint_as_float(w[i]);
        else if constexpr (VEC == 0) return __uint_as_float(w[i] << 16);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    // Rounds value i to nearest even; every i in ascending order.
    __device__ __forceinline__ void set(int i, float v) {
        uint32_t u = __float_as_uint(v);
        if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0x7FC00000u;
        if constexpr (ELT == Elt::FP32) w[i] = u;
        else if constexpr (VEC == 0) w[i] = bf16_rne(u);
        else if (i & 1) w[i / 2] |= bf16_rne(u) << 16;
        else w[i / 2] = bf16_rne(u);
    }
};

// Row r of a matrix of elements.
template <Elt ELT>
__device__ __forceinline__ const void* row_of(const void* p, int64_t r, int64_t ld) {
    return static_cast<const char*>(p) + r * ld * (ELT == Elt::BF16 ? 2 : 4);
}
template <Elt ELT>
__device__ __forceinline__ void* row_of(void* p, int64_t r, int64_t ld) {
    return static_cast<char*>(p) + r * ld * (ELT == Elt::BF16 ? 2 : 4);
}

// One row of the order to blockIdx.x, a slice of its pieces to blockIdx.y.
// Memory-bound: 32764 rows of 7184 bf16 139 us, 6.8 TB/s of what is read and
// written (a token is read for each of its choices; read once it would be 87).
template <Elt ELT, int VEC>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(MoeRowsArgs a) {
    let_next_start();
    wait_for_stream();
    using P = Piece<ELT, VEC, kRowThreads>;
    const int64_t pieces = P::count(a.H);
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x) {
        const int c = a.source[r];
        const int64_t t = c < 0 ? -1 : c / a.topk;
        const bool there = t >= 0 && t < a.T;
        for (int64_t i = (int64_t)blockIdx.y * kRowThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.y * kRowThreads) {
            P p;
            if (there)
                p.read(row_of<ELT>(a.tokens, t, a.ld_tokens), i, a.H);
            else
                p.clear();
            p.write(row_of<ELT>(a.out, r, a.H), i, a.H);
        }
    }
}

// out[t] = sum_j w_j y[slot_j]: one token to blockIdx.x, a slice of its pieces
// to blockIdx.y; the rows of four choices are loaded before they are added.
// Memory-bound; four blocks a multiprocessor, or the loads in flight do not
// suffice: 8191 tokens x 4 of 7184 bf16 88.6 us, 6.6 TB/s (three blocks 111).
template <Elt ELT, int VEC>
__global__ void __launch_bounds__(kRowThreads, 4) combine_kernel(MoeRowsArgs a) {
    let_next_start();
    wait_for_stream();
    using P = Piece<ELT, VEC, kRowThreads>;
    const int64_t pieces = P::count(a.H);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
        for (int64_t i = (int64_t)blockIdx.y * kRowThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.y * kRowThreads) {
            float sum[P::kValues] = {};
            for (int64_t j0 = 0; j0 < a.topk; j0 += kTogether) {
                P p[kTogether];
                bool there[kTogether];
                float w[kTogether];
#pragma unroll
                for (int j = 0; j < kTogether; ++j) {
                    const int64_t c = t * a.topk + j0 + j;
                    const int64_t r = j0 + j < a.topk ? a.slots[c] : -1;
                    there[j] = r >= 0 && r < a.R;
                    w[j] = there[j] && a.weights ? a.weights[c] : 1.0f;
                    if (there[j]) p[j].read(row_of<ELT>(a.rows, r, a.ld_rows), i, a.H);
                }
#pragma unroll
                for (int j = 0; j < kTogether; ++j)
                    if (there[j])
#pragma unroll
                        for (int q = 0; q < P::kValues; ++q) sum[q] = fmaf(w[j], p[j].at(q), sum[q]);
            }
            P o;
#pragma unroll
            for (int q = 0; q < P::kValues; ++q) o.set(q, sum[q]);
            o.write(row_of<ELT>(a.out, t, a.H), i, a.H);
        }
}

// TG choices of one token to a block.  The dot products are summed in a fixed
// order: a thread's pieces, the warp's lanes, the warps.  The blocks behind
// the tokens' clear the rows of no choice.  8191 tokens x 4 of 7184 bf16: 175
// us, 6.05 TB/s.  A piece's loads wait for the one before, and the block for
// its last thread: small blocks, 14 a multiprocessor, hide most of it (256
// threads 213 us, 128 192, 32 184), pieces of 16 bytes leave registers for that.
template <Elt ELT, int VEC, int TG, int THREADS>
__global__ void __launch_bounds__(THREADS, 896 / THREADS) combine_grad_kernel(MoeRowsArgs a, int64_t work, int64_t work_blocks) {
    let_next_start();
    wait_for_stream();
    using P = Piece<ELT, VEC, THREADS>;
    const int64_t pieces = P::count(a.H), n = a.T * a.topk;
    if (blockIdx.x >= work_blocks) {
        // each thread looks at one of the block's next rows; those of no choice are cleared by the whole block
        __shared__ int empty[THREADS];
        __shared__ int found;
        for (int64_t r0 = (blockIdx.x - work_blocks) * THREADS; r0 < a.R; r0 += (gridDim.x - work_blocks) * THREADS) {
            if (threadIdx.x == 0) found = 0;
            __syncthreads();
            const int64_t r = r0 + threadIdx.x;
            const int c = r < a.R ? a.source[r] : 0;
            if (c < 0 || c >= n) empty[atomicAdd(&found, 1)] = (int)threadIdx.x;
            __syncthreads();
            P zero;
            zero.clear();
            for (int x = 0; x < found; ++x)
                for (int64_t i = threadIdx.x; i < pieces; i += THREADS) zero.write(row_of<ELT>(a.out, r0 + empty[x], a.H), i, a.H);
            __syncthreads();
        }
        return;
    }
    __shared__ float part[THREADS / 32][TG];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t groups = (a.topk + TG - 1) / TG;
    for (int64_t x = blockIdx.x; x < work; x += work_blocks) {
        int64_t t, j0;
        split_index(x, groups, t, j0);
        j0 *= TG;
        float dot[TG] = {}, w[TG];
        int64_t row[TG];
#pragma unroll
        for (int j = 0; j < TG; ++j) {
            const int64_t c = t * a.topk + j0 + j;
            row[j] = j0 + j < a.topk ? a.slots[c] : -1;
            if (row[j] >= a.R) row[j] = -1;
            w[j] = row[j] >= 0 ? a.weights[c] : 0.0f;
        }
#pragma unroll 1
        for (int64_t i = threadIdx.x; i < pieces; i += THREADS) {
            P g, y[TG];
            g.read(row_of<ELT>(a.tokens, t, a.ld_tokens), i, a.H);
#pragma unroll
            for (int j = 0; j < TG; ++j)
                if (row[j] >= 0) y[j].read(row_of<ELT>(a.rows, row[j], a.ld_rows), i, a.H);
#pragma unroll
            for (int j = 0; j < TG; ++j)
                if (row[j] >= 0) {
                    P o;
#pragma unroll
                    for (int q = 0; q < P::kValues; ++q) {
                        dot[j] = fmaf(g.at(q), y[j].at(q), dot[j]);
                        o.set(q, w[j] * g.at(q));
                    }
                    o.write(row_of<ELT>(a.out, row[j], a.H), i, a.H);
                }
        }
#pragma unroll
        for (int j = 0; j < TG; ++j) {
#pragma unroll
            for (int d = 16; d; d /= 2) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
            if (lane == 0) part[warp][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < TG && j0 + threadIdx.x < a.topk) {
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < THREADS / 32; ++v) sum += part[v][threadIdx.x];
            a.d_weights[t * a.topk + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// Rows that begin on 32 bytes and hold whole pieces.
template <Elt ELT>
bool whole_pieces(const MoeRowsArgs& a) {
    constexpr int64_t es = ELT == Elt::BF16 ? 2 : 4;
    const auto on32 = [](const void* p, int64_t rows, int64_t bytes) {
        return reinterpret_cast<uintptr_t>(p) % 32 == 0 && (rows <= 1 || bytes % 32 == 0);
    };
    return a.H * es % 32 == 0 && on32(a.tokens, a.T, a.ld_tokens * es) && on32(a.rows, a.R, a.ld_rows * es) &&
           on32(a.out, 2, a.H * es);
}

constexpr int64_t kMostBlocks = INT64_C(0x7FFFFFFF);

// One row to a block; few rows are cut into slices so that the device is full.
dim3 row_grid(int64_t rows, int64_t pieces) {
    const int64_t slices = ceil_div(pieces, kRowThreads), wanted = ceil_div((int64_t)sm_count() * 8, rows);
    return dim3((unsigned)(rows < kMostBlocks ? rows : kMostBlocks),
                (unsigned)(wanted < 1 ? 1 : wanted < slices ? wanted : slices < 65535 ? slices : 65535));
}

template <Elt ELT, int VEC>
cudaError_t rows_launch(int what, const MoeRowsArgs& a, cudaStream_t s) {
    if (what == 0) {
        return launch_overlapped(dispatch_kernel<ELT, VEC>, row_grid(a.R, ceil_div(a.H, VEC ? VEC : 8)), kRowThreads, 0, 0, s, a);
    } else if (what == 1) {
        return launch_overlapped(combine_kernel<ELT, VEC>, row_grid(a.T, ceil_div(a.H, VEC ? VEC : 8)), kRowThreads, 0, 0, s, a);
    } else {
        // four choices to a block of 64 threads, or, where that leaves the device empty, one to a block of 128 (64 tokens of
        // 7184, topk 4, bf16: 4.7 us, 6.8 as the others; 8191 tokens: 282 us, 175 as the others)
        const bool few = a.T * ceil_div(a.topk, kTogether) < 8 * (int64_t)sm_count();
        const int64_t work = a.T * ceil_div(a.topk, few ? 1 : kTogether), work_blocks = work < (1 << 30) ? work : 1 << 30;
        const int64_t room = ceil_div(a.R, 64), clear = room < sm_count() ? room : sm_count();
        const dim3 grid((unsigned)(work_blocks + clear));
        constexpr int V = VEC / 2;
        return few ? launch_overlapped(combine_grad_kernel<ELT, V, 1, 128>, grid, 128, 0, 0, s, a, work, work_blocks)
                   : launch_overlapped(combine_grad_kernel<ELT, V, kTogether, 64>, grid, 64, 0, 0, s, a, work, work_blocks);
    }
}

cudaError_t rows_launch(int what, Elt elt, const MoeRowsArgs& a, cudaStream_t s) {
    const cudaError_t e =
        elt == Elt::BF16
            ? (whole_pieces<Elt::BF16>(a) ? rows_launch<Elt::BF16, 16>(what, a, s) : rows_launch<Elt::BF16, 0>(what, a, s))
            : (whole_pieces<Elt::FP32>(a) ? rows_launch<Elt::FP32, 8>(what, a, s) : rows_launch<Elt::FP32, 0>(what, a, s));
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace

int64_t moe_sort_chunks(int64_t choices) { return ceil_div(choices, kChunk); }

cudaError_t launch_moe_sort(const MoeSortArgs& a, cudaStream_t s) {
    const int chunks = (int)moe_sort_chunks(a.choices);
    // as many warps as have choices and as shared memory has room for histograms of
    const int threads = a.choices <= 1024 ? 256 : 1024;
    int walkers = kHistograms / ((int)a.experts * 4);
    walkers = walkers < threads / 32 ? walkers : threads / 32;
    const int one = (int)a.experts * 4, hist = walkers * one, place = hist + (int)(3 * a.experts + 1) * 4;
    static std::atomic<bool> allowed[kDevices];
    cudaError_t e = allow_shared_memory(place_kernel, kHistograms + (3 * kMostExperts + 1) * 4, allowed);
    if (e == cudaSuccess && chunks > 1) e = launch_overlapped(count_kernel, dim3(chunks), threads, one, 0, s, a, walkers);
    if (e == cudaSuccess) {
        // not overlapped with count_kernel: its blocks would take the multiprocessors' threads while that still runs
        // (65536 x 8 over 256 experts: 14.4 us; overlapped 20)
        place_kernel<<<chunks, threads, place, s>>>(a, chunks, walkers);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

cudaError_t launch_moe_dispatch(Elt elt, const MoeRowsArgs& a, cudaStream_t s) { return rows_launch(0, elt, a, s); }
cudaError_t launch_moe_combine(Elt elt, const MoeRowsArgs& a, cudaStream_t s) { return rows_launch(1, elt, a, s); }
cudaError_t launch_moe_combine_grad(Elt elt, const MoeRowsArgs& a, cudaStream_t s) { return rows_launch(2, elt, a, s); }

}  // namespace mxq
