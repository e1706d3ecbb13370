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

struct MoeFp8Args {
    const uint8_t* data;    // [T, ld]
    const uint8_t* scales;  // [T, nb]
    int64_t T, topk, R, K, nb, ld;
    const int32_t* source;
    uint8_t* out;         // [R, K]
    uint8_t* out_scales;  // [R, nb]
};

struct NormArgs {
    const void* x;
    const void* residual;  // optional
    const void* weight;
    Elt weight_elt;
    int64_t rows, K, ldx, ldr, ldh;
    float eps;
    void* h;          // optional, with a residual
    void* y;          // optional, contiguous
    uint8_t* data;    // optional, with scales
    uint8_t* scales;  // [rows, ceil(K/128)]
    float* rstd;      // optional
};

// Sums over rows that the blocks of the norm's gradient leave for its second
// kernel, at most: one of each block where they are persistent, one to a
// multiprocessor (152 on a GB300), and twice as many where rows are longer than
// those take.
constexpr int64_t kNormParts = 304;

struct NormGradArgs {
    const void *g, *h, *weight;
    Elt weight_elt;
    const float* rstd;
    const void* g_h;  // optional
    int64_t rows, K, ldg, ldh, ldgh, ldd;
    void* d_h;
    float* d_weight;  // optional, with parts
    float* parts;     // workspace [min(rows, kNormParts), K]
};

enum class GateForm { PLAIN, ROWS, COLUMNS, GRAD };

struct GateArgs {
    const void* x;  // [rows, ldx]: gate in columns 0..H-1, up in H..2H-1
    int64_t rows, H, ldx;
    const void* g;  // GRAD: [rows, ldg]
    int64_t ldg;
    void* out;        // PLAIN: [rows, H]; GRAD: [rows, 2H]
    uint8_t* data;    // ROWS, COLUMNS: [rows, H]
    uint8_t* scales;  // ROWS: [rows, ceil(H/128)]; COLUMNS: [ceil(rows/128), H]
};

struct RouteArgs {
    const void* logits;  // [T, ld]
    int64_t T, ld;
    int E, topk, groups, topk_groups, group_top;
    bool sigmoid, renorm;
    float scale;
    const float* bias;  // optional
    int32_t* ids;       // [T, topk]; the gradient reads them
    float* weights;     // [T, topk]
    const float* g;     // gradient: of the weights
    void* d_logits;     // gradient: [T, E]
    // set by the launcher: 16-byte accesses; experts of a group, and the binary logarithm of its lanes
    bool vector;
    int group_size, group_shift;
};

// Each returns cudaSuccess or the launch error.
cudaError_t launch_quant128(Elt elt, bool columns, const Quant128Args& a, cudaStream_t s);
cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t s);
cudaError_t launch_repack(const uint8_t* src, int64_t ld, int64_t rows, int64_t n, uint8_t* dst, int64_t ldd,
                          cudaStream_t s);
int64_t moe_sort_chunks(int64_t choices);
cudaError_t launch_moe_sort(const MoeSortArgs& a, cudaStream_t s);
cudaError_t launch_moe_dispatch(Elt elt, const MoeRowsArgs& a, cudaStream_t s);
cudaError_t launch_moe_dispatch_fp8(const MoeFp8Args& a, cudaStream_t s);
cudaError_t launch_norm(Elt elt, const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_grad(Elt elt, const NormGradArgs& a, cudaStream_t s);
cudaError_t launch_gate(Elt elt, GateForm form, const GateArgs& a, cudaStream_t s);
cudaError_t launch_route(Elt elt, bool grad, const RouteArgs& a, cudaStream_t s);
cudaError_t launch_moe_combine(Elt elt, const MoeRowsArgs& a, cudaStream_t s);
cudaError_t launch_moe_combine_grad(Elt elt, const MoeRowsArgs& a, cudaStream_t s);

}  // namespace mxq
