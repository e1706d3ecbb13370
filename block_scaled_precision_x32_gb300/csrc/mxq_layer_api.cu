// mxq_layer_api.cu -- C entry points of the FP8 linear layer and the
// mixture-of-experts operators: host-side argument checks, then the launches
// on the caller's stream.  Declared and documented in include/mxq.h.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mxq.h"
#include "mxq_layer.h"

namespace {

constexpr int64_t kMaxDim = INT64_C(0x7FFFFFFF);
constexpr int64_t kMaxLd = INT64_C(1) << 39;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

mxq_status check_dtype(mxq_dtype dt) {
    if (dt == MXQ_BF16 || dt == MXQ_FP32) return MXQ_OK;
    if (dt == MXQ_FP16) return MXQ_ERR_UNSUPPORTED_DTYPE;
    return MXQ_ERR_INVALID_ARG;
}

size_t elt_size(mxq_dtype dt) { return dt == MXQ_BF16 ? 2 : 4; }
mxq::Elt elt_of(mxq_dtype dt) { return dt == MXQ_BF16 ? mxq::Elt::BF16 : mxq::Elt::FP32; }
mxq_status launch_status(cudaError_t e) { return e == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA; }

bool valid_dim(int64_t n) { return n >= 0 && n <= kMaxDim; }
bool valid_width(int64_t n) { return n >= 0 && n <= (INT64_C(1) << 30); }  // of a row that is indexed in 32 bits
bool valid_ld(int64_t n, int64_t ld) { return ld >= n && ld <= kMaxLd; }

mxq_status quant128(bool columns, const void* x, mxq_dtype dt, int64_t rows, int64_t K, int64_t ldx,
                    const int32_t* index, int32_t index_div, int64_t out_rows, uint8_t* data, uint8_t* scales,
                    cudaStream_t stream) {
    const mxq_status st = check_dtype(dt);
    if (st != MXQ_OK) return st;
    if (!valid_dim(rows) || !valid_dim(K) || !valid_dim(out_rows) || !valid_ld(K, ldx)) return MXQ_ERR_INVALID_ARG;
    if (index ? index_div < 1 : out_rows != rows) return MXQ_ERR_INVALID_ARG;
    if (out_rows == 0 || K == 0) return MXQ_OK;
    if ((!x && rows > 0) || !data || !scales || !aligned(x, elt_size(dt))) return MXQ_ERR_INVALID_ARG;
    if (index && !aligned(index, 4)) return MXQ_ERR_INVALID_ARG;
    mxq::Quant128Args a{};
    a.x = x;
    a.rows = rows;
    a.K = K;
    a.ldx = ldx;
    a.index = index;
    a.index_div = index ? index_div : 1;
    a.out_rows = out_rows;
    a.data = data;
    a.scales = scales;
    return launch_status(mxq::launch_quant128(elt_of(dt), columns, a, stream));
}

// ---- the product: checks, then A and B in the kernels' terms

int64_t blocks(int64_t n) { return (n + 127) / 128; }
int64_t padded16(int64_t n) { return (n + 15) / 16 * 16; }

struct Operands {
    int64_t a_rows, a_n, b_rows, b_n;  // memory rows and bytes per row of a and b
    int64_t out_rows, out_n, E;
};

Operands operands(const mxq_fp8_product& p) {
    Operands o;
    o.E = p.offsets ? p.E : 1;
    o.a_rows = p.M;
    o.a_n = p.dir == MXQ_MATMUL_FWD ? p.K : p.N;
    o.b_rows = p.dir == MXQ_MATMUL_WGRAD ? p.M : o.E * p.N;
    o.b_n = p.K;
    o.out_rows = p.dir == MXQ_MATMUL_WGRAD ? p.N * o.E : p.M;
    o.out_n = p.dir == MXQ_MATMUL_FWD ? p.N : p.K;
    return o;
}

mxq_status check_product(const mxq_fp8_product* p) {
    if (!p) return MXQ_ERR_INVALID_ARG;
    if (p->dir != MXQ_MATMUL_FWD && p->dir != MXQ_MATMUL_DGRAD && p->dir != MXQ_MATMUL_WGRAD)
        return MXQ_ERR_INVALID_ARG;
    const mxq_status st = check_dtype(p->out_dt);
    if (st != MXQ_OK) return st;
    for (int64_t n : {p->M, p->N, p->K})
        if (n < 0 || n > (INT64_C(1) << 30)) return MXQ_ERR_INVALID_ARG;
    if (p->offsets && (p->E < 1 || p->E > 1024 || !aligned(p->offsets, 4))) return MXQ_ERR_INVALID_ARG;
    const Operands o = operands(*p);
    if (!valid_ld(o.a_n, p->lda) || !valid_ld(o.b_n, p->ldb) || !valid_ld(o.out_n, p->ldo)) return MXQ_ERR_INVALID_ARG;
    return MXQ_OK;
}

// TMA reads rows that start on 16 bytes.
bool needs_repack(const uint8_t* p, int64_t rows, int64_t ld) {
    return !aligned(p, 16) || (rows > 1 && ld % 16 != 0);
}

}  // namespace

extern "C" {

mxq_status mxq_fp8_quant_1x128(const void* x, mxq_dtype dt, int64_t rows, int64_t K, int64_t ldx, const int32_t* index,
                               int32_t index_div, int64_t out_rows, uint8_t* data, uint8_t* scales,
                               cudaStream_t stream) {
    return quant128(false, x, dt, rows, K, ldx, index, index_div, out_rows, data, scales, stream);
}

mxq_status mxq_fp8_quant_128x1(const void* x, mxq_dtype dt, int64_t rows, int64_t K, int64_t ldx, const int32_t* index,
                               int32_t index_div, int64_t out_rows, uint8_t* data, uint8_t* scales,
                               cudaStream_t stream) {
    return quant128(true, x, dt, rows, K, ldx, index, index_div, out_rows, data, scales, stream);
}

size_t mxq_fp8_matmul_workspace(const mxq_fp8_product* p) {
    if (check_product(p) != MXQ_OK) return 0;
    const Operands o = operands(*p);
    size_t n = 0;
    if (needs_repack(p->a, o.a_rows, p->lda)) n += (size_t)(o.a_rows * padded16(o.a_n));
    if (needs_repack(p->b, o.b_rows, p->ldb)) n += (size_t)(o.b_rows * padded16(o.b_n));
    return n;
}

mxq_status mxq_fp8_matmul(const mxq_fp8_product* p, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    mxq_status st = check_product(p);
    if (st != MXQ_OK) return st;
    const Operands o = operands(*p);
    if (o.out_rows == 0 || o.out_n == 0) return MXQ_OK;
    const size_t es = elt_size(p->out_dt);
    if (!p->out || !aligned(p->out, es)) return MXQ_ERR_INVALID_ARG;
    const int64_t depth = p->dir == MXQ_MATMUL_FWD ? p->K : p->dir == MXQ_MATMUL_DGRAD ? p->N : p->M;
    if (depth == 0)  // a sum of nothing
        return launch_status(cudaMemset2DAsync(p->out, (size_t)p->ldo * es, 0, (size_t)o.out_n * es,
                                               (size_t)o.out_rows, stream));
    if (!p->a || !p->b || !p->a_scales || !p->b_scales) return MXQ_ERR_INVALID_ARG;
    if (p->dir != MXQ_MATMUL_WGRAD && !aligned(p->b_scales, 4)) return MXQ_ERR_INVALID_ARG;
    const size_t need = mxq_fp8_matmul_workspace(p);
    if (need && (!workspace || workspace_bytes < need)) return MXQ_ERR_BUFFER_TOO_SMALL;
    if (need && !aligned(workspace, 16)) return MXQ_ERR_INVALID_ARG;

    const uint8_t *a = p->a, *b = p->b;
    int64_t lda = p->lda, ldb = p->ldb;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (needs_repack(a, o.a_rows, lda)) {
        lda = padded16(o.a_n);
        st = launch_status(mxq::launch_repack(a, p->lda, o.a_rows, o.a_n, ws, lda, stream));
        if (st != MXQ_OK) return st;
        a = ws;
        ws += o.a_rows * lda;
    }
    if (needs_repack(b, o.b_rows, ldb)) {
        ldb = padded16(o.b_n);
        st = launch_status(mxq::launch_repack(b, p->ldb, o.b_rows, o.b_n, ws, ldb, stream));
        if (st != MXQ_OK) return st;
        b = ws;
    }

    mxq::MatmulArgs g{};
    g.a.data = a;
    g.a.ld = lda;
    g.a.scales = p->a_scales;
    g.b.data = b;
    g.b.ld = ldb;
    g.b.scales = p->b_scales;
    g.depth = depth;
    g.out = p->out;
    g.out_bf16 = p->out_dt == MXQ_BF16;
    g.ldo = p->ldo;
    g.offsets = p->offsets;
    g.E = p->offsets ? p->E : 0;
    g.grouping = !p->offsets ? mxq::Grouping::NONE
                             : p->dir == MXQ_MATMUL_WGRAD ? mxq::Grouping::DEPTH : mxq::Grouping::ROWS;
    if (p->dir == MXQ_MATMUL_WGRAD) {
        g.a.rows = p->N;
        g.a.mn = true;
        g.a.s_row = 1;
        g.a.s_kb = p->N;
        g.b.rows = p->K;
        g.b.mn = true;
        g.b.s_row = 1;
        g.b.s_kb = p->K;
        g.out_expert = p->N * p->ldo;
    } else {
        const int64_t nt = blocks(p->N), kt = blocks(p->K);
        g.a.rows = p->M;
        g.a.s_row = blocks(depth);
        g.a.s_kb = 1;
        g.b.tiles = true;
        g.b.rows = p->dir == MXQ_MATMUL_FWD ? p->N : p->K;
        g.b.mn = p->dir == MXQ_MATMUL_DGRAD;
        g.b.s_row = p->dir == MXQ_MATMUL_FWD ? kt : 1;
        g.b.s_kb = p->dir == MXQ_MATMUL_FWD ? 1 : kt;
        if (p->offsets) {
            g.b.expert = p->N * ldb;
            g.b.s_expert = nt * kt;
        }
    }
    return launch_status(mxq::launch_matmul(g, stream));
}

int64_t mxq_moe_capacity(int64_t tokens, int64_t topk, int64_t experts, int64_t align) {
    if (tokens <= 0 || topk <= 0 || experts <= 0 || align <= 0) return 0;
    const int64_t n = tokens * topk;
    return n + (experts < n ? experts : n) * (align - 1);
}

size_t mxq_moe_sort_workspace(int64_t tokens, int64_t topk, int64_t experts) {
    if (tokens <= 0 || topk <= 0 || experts <= 0) return 0;
    const int64_t chunks = mxq::moe_sort_chunks(tokens * topk);
    return chunks > 1 ? (size_t)(chunks * experts * 4) : 0;
}

mxq_status mxq_moe_sort(const int32_t* ids, int64_t tokens, int64_t topk, int64_t experts, int64_t align,
                        int32_t* offsets, int32_t* source, int32_t* slots, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
    if (!valid_dim(tokens) || !valid_dim(topk) || experts < 1 || experts > 2048 || align < 1 || align > kMaxDim)
        return MXQ_ERR_INVALID_ARG;
    if (topk > 0 && tokens > kMaxDim / topk) return MXQ_ERR_INVALID_ARG;
    const int64_t n = tokens * topk, cap = mxq_moe_capacity(tokens, topk, experts, align);
    if (cap > kMaxDim) return MXQ_ERR_INVALID_ARG;
    if (!offsets || !aligned(offsets, 4)) return MXQ_ERR_INVALID_ARG;
    if (n > 0 && (!ids || !source || !slots || !aligned(ids, 4) || !aligned(source, 4) || !aligned(slots, 4)))
        return MXQ_ERR_INVALID_ARG;
    if (n == 0) return launch_status(cudaMemsetAsync(offsets, 0, (size_t)(experts + 1) * 4, stream));
    const size_t need = mxq_moe_sort_workspace(tokens, topk, experts);
    if (need && (!workspace || workspace_bytes < need)) return MXQ_ERR_BUFFER_TOO_SMALL;
    if (need && !aligned(workspace, 4)) return MXQ_ERR_INVALID_ARG;
    mxq::MoeSortArgs a{};
    a.ids = ids;
    a.choices = n;
    a.experts = experts;
    a.align = align;
    a.capacity = cap;
    a.offsets = offsets;
    a.source = source;
    a.slots = slots;
    a.counts = static_cast<int32_t*>(workspace);
    return launch_status(mxq::launch_moe_sort(a, stream));
}

mxq_status mxq_moe_dispatch(const void* x, mxq_dtype dt, int64_t tokens, int64_t H, int64_t ldx, const int32_t* source,
                            int64_t topk, int64_t rows, void* out, cudaStream_t stream) {
    const mxq_status st = check_dtype(dt);
    if (st != MXQ_OK) return st;
    if (!valid_dim(tokens) || !valid_dim(H) || !valid_dim(rows) || !valid_ld(H, ldx) || topk < 1 || topk > kMaxDim)
        return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || H == 0) return MXQ_OK;
    if ((!x && tokens > 0) || !source || !out || !aligned(x, elt_size(dt)) || !aligned(out, elt_size(dt)) ||
        !aligned(source, 4))
        return MXQ_ERR_INVALID_ARG;
    mxq::MoeRowsArgs a{};
    a.tokens = x;
    a.T = tokens;
    a.topk = topk;
    a.R = rows;
    a.H = H;
    a.ld_tokens = ldx;
    a.source = source;
    a.out = out;
    return launch_status(mxq::launch_moe_dispatch(elt_of(dt), a, stream));
}

mxq_status mxq_moe_combine(const void* y, mxq_dtype dt, int64_t rows, int64_t H, int64_t ldy, const int32_t* slots,
                           const float* weights, int64_t tokens, int64_t topk, void* out, cudaStream_t stream) {
    const mxq_status st = check_dtype(dt);
    if (st != MXQ_OK) return st;
    if (!valid_dim(tokens) || !valid_dim(H) || !valid_dim(rows) || !valid_ld(H, ldy) || topk < 0 || topk > kMaxDim)
        return MXQ_ERR_INVALID_ARG;
    if (tokens == 0 || H == 0) return MXQ_OK;
    if ((!y && rows > 0) || (!slots && topk > 0) || !out || !aligned(y, elt_size(dt)) || !aligned(out, elt_size(dt)) ||
        !aligned(slots, 4) || !aligned(weights, 4))
        return MXQ_ERR_INVALID_ARG;
    mxq::MoeRowsArgs a{};
    a.rows = y;
    a.T = tokens;
    a.topk = topk;
    a.R = rows;
    a.H = H;
    a.ld_rows = ldy;
    a.slots = slots;
    a.weights = weights;
    a.out = out;
    return launch_status(mxq::launch_moe_combine(elt_of(dt), a, stream));
}

mxq_status mxq_moe_combine_grad(const void* g, const void* y, mxq_dtype dt, int64_t tokens, int64_t topk, int64_t rows,
                                int64_t H, int64_t ldg, int64_t ldy, const int32_t* source, const int32_t* slots,
                                const float* weights, void* d_rows, float* d_weights, cudaStream_t stream) {
    const mxq_status st = check_dtype(dt);
    if (st != MXQ_OK) return st;
    if (!valid_dim(tokens) || !valid_dim(H) || !valid_dim(rows) || !valid_ld(H, ldg) || !valid_ld(H, ldy) || topk < 0 ||
        topk > kMaxDim || (topk > 0 && tokens > kMaxDim / topk))
        return MXQ_ERR_INVALID_ARG;
    const int64_t n = tokens * topk;
    const size_t es = elt_size(dt);
    if (n > 0 && (!slots || !weights || !d_weights || !aligned(slots, 4) || !aligned(weights, 4) ||
                  !aligned(d_weights, 4)))
        return MXQ_ERR_INVALID_ARG;
    if (H == 0)  // dot products of nothing
        return n ? launch_status(cudaMemsetAsync(d_weights, 0, (size_t)n * 4, stream)) : MXQ_OK;
    if (n == 0 && rows == 0) return MXQ_OK;
    if ((tokens > 0 && !g) || (rows > 0 && (!y || !d_rows || !source)) || !aligned(g, es) || !aligned(y, es) ||
        !aligned(d_rows, es) || !aligned(source, 4))
        return MXQ_ERR_INVALID_ARG;
    mxq::MoeRowsArgs a{};
    a.tokens = g;
    a.rows = y;
    a.T = tokens;
    a.topk = topk;
    a.R = rows;
    a.H = H;
    a.ld_tokens = ldg;
    a.ld_rows = ldy;
    a.source = source;
    a.slots = slots;
    a.weights = weights;
    a.out = d_rows;
    a.d_weights = d_weights;
    return launch_status(mxq::launch_moe_combine_grad(elt_of(dt), a, stream));
}

mxq_status mxq_fp8_dispatch(const uint8_t* data, const uint8_t* scales, int64_t tokens, int64_t K, int64_t ld,
                            const int32_t* source, int64_t topk, int64_t rows, uint8_t* out, uint8_t* out_scales,
                            cudaStream_t stream) {
    if (!valid_dim(tokens) || !valid_width(K) || !valid_dim(rows) || !valid_ld(K, ld) || topk < 1 || topk > kMaxDim)
        return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return MXQ_OK;
    if ((tokens > 0 && (!data || !scales)) || !source || !out || !out_scales || !aligned(source, 4)) return MXQ_ERR_INVALID_ARG;
    mxq::MoeFp8Args a{};
    a.data = data;
    a.scales = scales;
    a.T = tokens;
    a.topk = topk;
    a.R = rows;
    a.K = K;
    a.nb = blocks(K);
    a.ld = ld;
    a.source = source;
    a.out = out;
    a.out_scales = out_scales;
    return launch_status(mxq::launch_moe_dispatch_fp8(a, stream));
}

// ---- the norm

mxq_status mxq_rmsnorm(const mxq_norm* p, cudaStream_t stream) {
    if (!p) return MXQ_ERR_INVALID_ARG;
    mxq_status st = check_dtype(p->dt);
    if (st != MXQ_OK) return st;
    st = check_dtype(p->weight_dt);
    if (st != MXQ_OK) return st;
    if (!valid_dim(p->rows) || !valid_width(p->K) || !valid_ld(p->K, p->ldx) || !(p->eps >= 0.0f && p->eps <= 3.4e38f))
        return MXQ_ERR_INVALID_ARG;
    if ((p->residual && !valid_ld(p->K, p->ldr)) || (p->h && (!p->residual || !valid_ld(p->K, p->ldh))) || !p->data != !p->scales)
        return MXQ_ERR_INVALID_ARG;
    if (p->rows == 0) return MXQ_OK;
    if (p->K == 0)  // the mean of nothing
        return p->rstd ? launch_status(cudaMemsetAsync(p->rstd, 0xFF, (size_t)p->rows * 4, stream)) : MXQ_OK;
    const size_t es = elt_size(p->dt);
    if (!p->x || !p->weight || !aligned(p->x, es) || !aligned(p->residual, es) || !aligned(p->weight, elt_size(p->weight_dt)) ||
        !aligned(p->h, es) || !aligned(p->y, es) || !aligned(p->rstd, 4))
        return MXQ_ERR_INVALID_ARG;
    // in place: the same rows
    if (p->rows > 1 && ((p->h == p->x && p->h && p->ldh != p->ldx) || (p->h && p->h == p->residual && p->ldh != p->ldr)))
        return MXQ_ERR_INVALID_ARG;
    if (!p->h && !p->y && !p->data && !p->rstd) return MXQ_OK;
    mxq::NormArgs a{};
    a.x = p->x;
    a.residual = p->residual;
    a.weight = p->weight;
    a.weight_elt = elt_of(p->weight_dt);
    a.rows = p->rows;
    a.K = p->K;
    a.ldx = p->ldx;
    a.ldr = p->ldr;
    a.ldh = p->ldh;
    a.eps = p->eps;
    a.h = p->h;
    a.y = p->y;
    a.data = p->data;
    a.scales = p->scales;
    a.rstd = p->rstd;
    return launch_status(mxq::launch_norm(elt_of(p->dt), a, stream));
}

size_t mxq_rmsnorm_grad_workspace(int64_t rows, int64_t K) {
    if (!valid_dim(rows) || !valid_width(K)) return 0;
    return (size_t)((rows < mxq::kNormParts ? rows : mxq::kNormParts) * K) * 4;
}

mxq_status mxq_rmsnorm_grad(const mxq_norm_grad* p, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!p) return MXQ_ERR_INVALID_ARG;
    mxq_status st = check_dtype(p->dt);
    if (st != MXQ_OK) return st;
    st = check_dtype(p->weight_dt);
    if (st != MXQ_OK) return st;
    if (!valid_dim(p->rows) || !valid_width(p->K) || !valid_ld(p->K, p->ldg) || !valid_ld(p->K, p->ldh) ||
        (p->g_h && !valid_ld(p->K, p->ldgh)) || !valid_ld(p->K, p->ldd) || !aligned(p->d_weight, 4))
        return MXQ_ERR_INVALID_ARG;
    if (p->K == 0) return MXQ_OK;
    if (p->rows == 0)
        return p->d_weight ? launch_status(cudaMemsetAsync(p->d_weight, 0, (size_t)p->K * 4, stream)) : MXQ_OK;
    const size_t es = elt_size(p->dt);
    if (!p->g || !p->h || !p->weight || !p->rstd || !p->d_h || !aligned(p->g, es) || !aligned(p->h, es) ||
        !aligned(p->weight, elt_size(p->weight_dt)) || !aligned(p->rstd, 4) || !aligned(p->g_h, es) || !aligned(p->d_h, es))
        return MXQ_ERR_INVALID_ARG;
    if (p->rows > 1 && ((p->d_h == p->g && p->ldd != p->ldg) || (p->d_h == p->h && p->ldd != p->ldh) ||
                        (p->d_h == p->g_h && p->ldd != p->ldgh)))
        return MXQ_ERR_INVALID_ARG;
    const size_t need = p->d_weight ? mxq_rmsnorm_grad_workspace(p->rows, p->K) : 0;
    if (need && (!workspace || workspace_bytes < need)) return MXQ_ERR_BUFFER_TOO_SMALL;
    if (need && !aligned(workspace, 16)) return MXQ_ERR_INVALID_ARG;
    mxq::NormGradArgs a{};
    a.g = p->g;
    a.h = p->h;
    a.weight = p->weight;
    a.weight_elt = elt_of(p->weight_dt);
    a.rstd = p->rstd;
    a.g_h = p->g_h;
    a.rows = p->rows;
    a.K = p->K;
    a.ldg = p->ldg;
    a.ldh = p->ldh;
    a.ldgh = p->ldgh;
    a.ldd = p->ldd;
    a.d_h = p->d_h;
    a.d_weight = p->d_weight;
    a.parts = need ? static_cast<float*>(workspace) : nullptr;
    return launch_status(mxq::launch_norm_grad(elt_of(p->dt), a, stream));
}

// ---- the gated activation

static mxq_status gate(mxq::GateForm form, const void* x, mxq_dtype dt, int64_t rows, int64_t H, int64_t ldx, const void* g, int64_t ldg,
                       void* out, uint8_t* data, uint8_t* scales, cudaStream_t stream) {
    const mxq_status st = check_dtype(dt);
    if (st != MXQ_OK) return st;
    const bool grad = form == mxq::GateForm::GRAD, quant = form == mxq::GateForm::ROWS || form == mxq::GateForm::COLUMNS;
    if (!valid_dim(rows) || !valid_width(H) || !valid_width(2 * H) || !valid_ld(2 * H, ldx) || (grad && !valid_ld(H, ldg))) return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || H == 0) return MXQ_OK;
    const size_t es = elt_size(dt);
    if (!x || !aligned(x, es) || (grad && (!g || !aligned(g, es)))) return MXQ_ERR_INVALID_ARG;
    if (quant ? (!data || !scales) : (!out || !aligned(out, es))) return MXQ_ERR_INVALID_ARG;
    mxq::GateArgs a{};
    a.x = x;
    a.rows = rows;
    a.H = H;
    a.ldx = ldx;
    a.g = g;
    a.ldg = ldg;
    a.out = out;
    a.data = data;
    a.scales = scales;
    return launch_status(mxq::launch_gate(elt_of(dt), form, a, stream));
}

mxq_status mxq_silu_mul(const void* x, mxq_dtype dt, int64_t rows, int64_t H, int64_t ldx, void* out, cudaStream_t stream) {
    return gate(mxq::GateForm::PLAIN, x, dt, rows, H, ldx, nullptr, 0, out, nullptr, nullptr, stream);
}

mxq_status mxq_fp8_silu_mul_1x128(const void* x, mxq_dtype dt, int64_t rows, int64_t H, int64_t ldx, uint8_t* data,
                                  uint8_t* scales, cudaStream_t stream) {
    return gate(mxq::GateForm::ROWS, x, dt, rows, H, ldx, nullptr, 0, nullptr, data, scales, stream);
}

mxq_status mxq_fp8_silu_mul_128x1(const void* x, mxq_dtype dt, int64_t rows, int64_t H, int64_t ldx, uint8_t* data,
                                  uint8_t* scales, cudaStream_t stream) {
    return gate(mxq::GateForm::COLUMNS, x, dt, rows, H, ldx, nullptr, 0, nullptr, data, scales, stream);
}

mxq_status mxq_silu_mul_grad(const void* g, const void* x, mxq_dtype dt, int64_t rows, int64_t H, int64_t ldg, int64_t ldx,
                             void* d_x, cudaStream_t stream) {
    return gate(mxq::GateForm::GRAD, x, dt, rows, H, ldx, g, ldg, d_x, nullptr, nullptr, stream);
}

// ---- the router

static bool valid_route(int64_t tokens, int64_t experts, int64_t ld, int64_t topk, int score, float scale) {
    return valid_dim(tokens) && experts >= 1 && experts <= 1024 && valid_ld(experts, ld) && topk >= 1 && topk <= 32 && topk <= experts &&
           tokens <= kMaxDim / topk && (score == MXQ_SCORE_SOFTMAX || score == MXQ_SCORE_SIGMOID) && scale >= -3.4e38f && scale <= 3.4e38f;
}

mxq_status mxq_moe_route(const mxq_route* p, int32_t* ids, float* weights, cudaStream_t stream) {
    if (!p) return MXQ_ERR_INVALID_ARG;
    const mxq_status st = check_dtype(p->dt);
    if (st != MXQ_OK) return st;
    if (!valid_route(p->tokens, p->experts, p->ld, p->topk, p->score, p->scale)) return MXQ_ERR_INVALID_ARG;
    if (p->groups < 1 || p->groups > 32 || p->experts % p->groups || p->topk_groups < 1 || p->topk_groups > p->groups || p->group_top < 1 ||
        p->group_top > 2 || p->group_top > p->experts / p->groups || p->topk > p->topk_groups * (p->experts / p->groups))
        return MXQ_ERR_INVALID_ARG;
    if (p->tokens == 0) return MXQ_OK;
    if (!p->logits || !aligned(p->logits, elt_size(p->dt)) || !aligned(p->bias, 4) || !ids || !aligned(ids, 4) || !weights ||
        !aligned(weights, 4))
        return MXQ_ERR_INVALID_ARG;
    mxq::RouteArgs a{};
    a.logits = p->logits;
    a.T = p->tokens;
    a.ld = p->ld;
    a.E = (int)p->experts;
    a.topk = (int)p->topk;
    a.groups = (int)p->groups;
    a.topk_groups = (int)p->topk_groups;
    a.group_top = (int)p->group_top;
    a.sigmoid = p->score == MXQ_SCORE_SIGMOID;
    a.renorm = p->renormalize != 0;
    a.scale = p->scale;
    a.bias = p->bias;
    a.ids = ids;
    a.weights = weights;
    return launch_status(mxq::launch_route(elt_of(p->dt), false, a, stream));
}

mxq_status mxq_moe_route_grad(const float* g, const mxq_route* p, const int32_t* ids, void* d_logits, cudaStream_t stream) {
    if (!p) return MXQ_ERR_INVALID_ARG;
    const mxq_status st = check_dtype(p->dt);
    if (st != MXQ_OK) return st;
    if (!valid_route(p->tokens, p->experts, p->ld, p->topk, p->score, p->scale)) return MXQ_ERR_INVALID_ARG;
    if (p->tokens == 0) return MXQ_OK;
    const size_t es = elt_size(p->dt);
    if (!g || !aligned(g, 4) || !p->logits || !aligned(p->logits, es) || !ids || !aligned(ids, 4) || !d_logits || !aligned(d_logits, es))
        return MXQ_ERR_INVALID_ARG;
    mxq::RouteArgs a{};
    a.logits = p->logits;
    a.T = p->tokens;
    a.ld = p->ld;
    a.E = (int)p->experts;
    a.topk = (int)p->topk;
    a.sigmoid = p->score == MXQ_SCORE_SIGMOID;
    a.renorm = p->renormalize != 0;
    a.scale = p->scale;
    a.ids = const_cast<int32_t*>(ids);
    a.g = g;
    a.d_logits = d_logits;
    return launch_status(mxq::launch_route(elt_of(p->dt), true, a, stream));
}

}  // extern "C"
