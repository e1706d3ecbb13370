// mxq_internal.h -- host-side launchers shared between the C entry points
// (mxq_api.cu) and the kernel translation units.  Not part of the ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime_api.h>

namespace mxq {

enum class Elt { BF16, FP32 };
enum class RowMode { PROJECT, MXFP8, MXFP4 };

struct RowwiseArgs {
    const void* x;
    void* y;          // PROJECT output
    uint8_t* data;    // MXFP8 payload [rows, K]; MXFP4 nibbles [rows, ceil(K/2)]
    uint8_t* scales;  // UE8M0 scale bytes in `lay`
    int64_t rows, K, ldx, ldy;
    int lay;          // mxq_scale_layout
    const int32_t* skip;  // optional device flag: nonzero = write nothing
};

struct Block128Args {
    const void* x;
    uint8_t* data;
    float* tile_scale_inv;
    int64_t rows, K, ldx;
    const int32_t* skip;  // optional device flag: nonzero = write nothing
};

struct ColwiseArgs {
    const void* x;
    uint8_t* data;    // [rows, K] E4M3
    uint8_t* scales;  // transposed scale matrix (K x ceil(rows/32)) in `lay`
    int64_t rows, K, ldx;
    int lay;
    const int32_t* skip;  // optional device flag: nonzero = write nothing
};

struct DequantArgs {
    int kind;  // mxq_quant_kind (0 MXFP8 row, 1 128x128, 2 packed MXFP4, 3 MXFP8 columnwise)
    const uint8_t* data;
    int64_t rows, K;
    int fp8;   // mxq_fp8
    const uint8_t* scales;
    int lay;
    const float* tile_scale_inv;
    void* out;
    bool out_bf16;
};

struct ExportArgs {
    const uint8_t* scales;
    int lay;
    int path;  // grouped export only: 1 = the chunk kernel's path (set by the launcher)
    int64_t rows, K;
    uint8_t* out;  // compact [rows, nb]
};

// Descriptors of a grouped export, passed by value as kernel parameters.
constexpr int kGroupedMax = 128;
struct GroupedExport {
    ExportArgs item[kGroupedMax];
    int count;
};

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
cudaError_t launch_rowwise(RowMode mode, Elt elt, const RowwiseArgs& a, cudaStream_t s);
cudaError_t launch_block128(Elt elt, const Block128Args& a, cudaStream_t s);
cudaError_t launch_dequant(const DequantArgs& a, cudaStream_t s);
cudaError_t launch_export(const ExportArgs& a, cudaStream_t s);
cudaError_t launch_export_grouped(const GroupedExport& b, cudaStream_t s);
cudaError_t launch_colwise(Elt elt, const ColwiseArgs& a, cudaStream_t s);
cudaError_t launch_colwise_dequant(const DequantArgs& a, cudaStream_t s);

cudaError_t launch_quant128(Elt elt, bool columns, const Quant128Args& a, cudaStream_t s);
cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t s);
cudaError_t launch_repack(const uint8_t* src, int64_t ld, int64_t rows, int64_t n, uint8_t* dst, int64_t ldd,
                          cudaStream_t s);
int64_t moe_sort_chunks(int64_t choices);
cudaError_t launch_moe_sort(const MoeSortArgs& a, cudaStream_t s);
cudaError_t launch_moe_dispatch(Elt elt, const MoeRowsArgs& a, cudaStream_t s);
cudaError_t launch_moe_combine(Elt elt, const MoeRowsArgs& a, cudaStream_t s);
cudaError_t launch_moe_combine_grad(Elt elt, const MoeRowsArgs& a, cudaStream_t s);

// Resident-grid sizing: number of SMs of the current device (cached).
int sm_count();

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace mxq
