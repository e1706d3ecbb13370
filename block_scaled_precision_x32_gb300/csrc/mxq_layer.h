// mxq_layer.h -- host-side launchers of the FP8 linear layer and the mixture of
// experts, shared between their C entry points (mxq_layer_api.cu) and their
// kernels.  Not part of the ABI.
#pragma once

#include "mxq_internal.h"

namespace mxq {

struct Quant128Args {
    const void* x;
    int64_t rows, K, ldx;
    const int32_t* index;  // optional: output row i is x row index[i] / index_div
    int32_t index_div;
    int64_t out_rows;
    uint8_t* data;    // [out_rows, K]
    uint8_t* scales;  // 1x128: [out_rows, ceil(K/128)]; 128x1: [ceil(out_rows/128), K]
};

// One operand of a product out[i, j] = sum_k A[i, k] B[j, k].  Element (i, k) is byte i*ld + k, or
// k*ld + i when `mn` (the index that survives the product runs along the memory's rows).
struct MatOperand {
    const uint8_t* data;
    int64_t rows;    // extent of i (or j)
    int64_t ld;
    bool mn;
    bool tiles;      // scales: fp32 per 128x128 tile, else a UE8M0 byte per element of i and 128-block of k
    const void* scales;
    int64_t s_row;   // stride of the scales along i (tiles: along i/128)
    int64_t s_kb;    // stride along k/128
    int64_t expert;  // byte stride of `data` from one expert's operand to the next (0: shared)
    int64_t s_expert;
};

enum class Grouping { NONE, ROWS, DEPTH };  // offsets cut up the rows of A, or the depth

struct MatmulArgs {
    MatOperand a, b;
    int64_t depth;
    Grouping grouping;
    const int32_t* offsets;
    int64_t E;
    void* out;
    bool out_bf16;
    int64_t ldo;
    int64_t out_expert;  // elements from one expert's output to the next (DEPTH)
};

struct MoeSortArgs {
    const int32_t* ids;
    int64_t choices, experts, align, capacity;
    int32_t *offsets, *source, *slots;
    int32_t* counts;  // workspace: [chunks, experts]
};

struct MoeRowsArgs {
    const void* tokens;  // x or g [T, ld_tokens]
    const void* rows;    // y [R, ld_rows]
    int64_t T, topk, R, H, ld_tokens, ld_rows;
    const int32_t *source, *slots;
    const float* weights;
    void* out;         // contiguous
    float* d_weights;  // combine's gradient only
};

// Each returns cudaSuccess or the launch error.
cudaError_t launch_quant128(Elt elt, bool columns, const Quant128Args& a, cudaStream_t s);
cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t s);
cudaError_t launch_repack(const uint8_t* src, int64_t ld, int64_t rows, int64_t n, uint8_t* dst, int64_t ldd,
                          cudaStream_t s);
int64_t moe_sort_chunks(int64_t choices);
cudaError_t launch_moe_sort(const MoeSortArgs& a, cudaStream_t s);
cudaError_t launch_moe_dispatch(Elt elt, const MoeRowsArgs& a, cudaStream_t s);
cudaError_t launch_moe_combine(Elt elt, const MoeRowsArgs& a, cudaStream_t s);
cudaError_t launch_moe_combine_grad(Elt elt, const MoeRowsArgs& a, cudaStream_t s);

}  // namespace mxq
