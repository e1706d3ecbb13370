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

// exp(-x) passes the end of fp32's range for a gate x of -87.3, but what it
// leaves of a large other factor may be any number.  Gates below kFar take it as
// exp(-x) 2^-116, and the other factor times 2^-116 as well, both exact: their
// results keep all their bits down to -167.7.  Below that they are 0, for what is
// less than 167.8 2^-242 = 2.4e-71 of the other factor.  (What the
// scaled factor loses where it is subnormal does not count: below kFar
// 2^116 x / (1 + exp(-x)), which it is multiplied with, is at most 1.)
constexpr float kFar = -85.0f, kShift = 116.0f, kScale = 0x1p-116f;
struct Scaled {
    float2 shift, scale;
    __device__ __forceinline__ explicit Scaled(float2 x) {
        const bool a = x.x < kFar, b = x.y < kFar;
        shift = make_float2(a ? kShift : 0.0f, b ? kShift : 0.0f);
        scale = make_float2(a ? kScale : 1.0f, b ? kScale : 1.0f);
    }
};

// 1 is added to it, or 2^-116 to what is larger: nothing is lost by taking
// subnormal results as zeros, which saves three instructions.
__device__ __forceinline__ float ex2_ftz(float t) {
    float p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
    return p;
}
__device__ __forceinline__ float2 ex2_neg(float2 t) { return make_float2(ex2_ftz(-t.x), ex2_ftz(-t.y)); }

// exp(-x) scale of two gates, off by 4 units of 2^-24 of itself: as exp_neg, for
// numbers of either sign.  CUT: that of -168, where 1 / (1 + exp(-x)) is 0, below it,
// and 0 above 160.  Else it passes into infinity, and is NaN for +inf.
//
// That of a bf16 gate takes fewer instructions: log2(e) is cut into K1 of 16 bits,
// whose product with the gate's 8 is exact, and the rest K2 = 7.1e-6: exp(-x) =
// 2^(-x K1) (1 - x K2 ln 2), off by (x K2 ln 2)^2 / 2 more for the second order left out,
// 1.5 units at 88 and 6 at 168.
template <Elt ELT, bool CUT>
__device__ __forceinline__ float2 exp_scaled(float2 x, const Scaled& c) {
    const auto cut = [](float v) {
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(-168.0f));
        return min_nan(v, kExpEnd);
    };
    if constexpr (CUT) x = make_float2(cut(x.x), cut(x.y));
    if constexpr (ELT == Elt::BF16) {
        constexpr float K1 = 47274.0f / 32768.0f, K2 = 7.0526077e-6f * kLn2;
        return mul2(ex2_neg(fma2(x, both(K1), c.shift)), fma2(x, both(-K2), both(1.0f)));
    } else {
        static_assert(CUT);  // the largest numbers' product with log2(e) is infinite
        const float2 t = mul2(x, both(-kExpHi)), r = fma2(x, both(kExpLo), fma2(x, both(kExpHi), t)), p = ex2_neg(fma2(t, both(1.0f), c.shift));
        return fma2(mul2(p, both(kLn2)), r, p);
    }
}

// N = 2, 4, ... values of a: gate and up as Unit's words hold them.  Bound by
// instructions as much as by memory, so two values go through each.
//
// silu(x) is taken as x / (1 + exp(-x)), which needs no choice by the sign; -inf
// gives the NaN that it has by its definition, 0 * inf.  In the FP8 forms an infinite
// bf16 gate gives NaN, of either sign: its block is poisoned as it would be by an
// infinity.
template <Elt ELT, int N, bool QUANT>
__device__ __forceinline__ void gated(const uint32_t* gate, const uint32_t* up, float* v) {
    const auto two = [](const uint32_t* w, int j) {
        if constexpr (ELT == Elt::BF16) return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
        else return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    };
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        const float2 x = two(gate, j);
        const Scaled c(x);
        const float2 d = fma2(exp_scaled<ELT, !QUANT || ELT == Elt::FP32>(x, c), both(1.0f), c.scale);
        const float2 r = mul2(mul2(x, make_float2(rcp_approx(d.x), rcp_approx(d.y))), mul2(two(up, j), c.scale));
        v[2 * j] = r.x, v[2 * j + 1] = r.y;
    }
}

// The same for elements that came one by one, as load_f32 leaves them.
template <Elt ELT, int N, bool QUANT>
__device__ __forceinline__ void gated_loose(const uint32_t* gate, const uint32_t* up, float* v) {
    if constexpr (ELT == Elt::BF16) {
        uint32_t g[N / 2], u[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            g[j] = prmt(gate[2 * j], gate[2 * j + 1], 0x7632u);
            u[j] = prmt(up[2 * j], up[2 * j + 1], 0x7632u);
        }
        gated<ELT, N, QUANT>(g, u, v);
    } else {
        gated<ELT, N, QUANT>(gate, up, v);
    }
}

// 2, 4 or a multiple of 8 words.
template <int W>
__device__ __forceinline__ void load_words(uint32_t* w, const char* p) {
    if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < W; j += 8) ld32(*reinterpret_cast<uint32_t(*)[8]>(w + j), p + 4 * j);
    }
}

// Largest magnitude of N values, as a pattern; above 0x7F800000 for a NaN among them.
template <int N>
__device__ __forceinline__ uint32_t amax_of(const float* v) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j += 2) m = absmax3(m, v[j], v[j + 1]);
    return __float_as_uint(m) & 0x7FFFFFFFu;
}

// Rows of units of 16 elements, eight lanes to a 1x128 block.  Bound by HBM:
// 16384 x 4096 bf16 to FP8 54.0 us, 6.2 TB/s (units of 8 elements 67 to 86; six or
// seven blocks a multiprocessor, whose registers spill, 59), to bf16 58.1, 6.9 TB/s.
template <Elt ELT, bool QUANT>
__global__ void __launch_bounds__(256, ELT == Elt::FP32 ? 4 : QUANT ? 5 : 6) gate_rows_kernel(GateArgs a, int64_t nb) {
    let_next_start();
    wait_for_stream();
    constexpr int N = 16, LANES = 128 / N, W = N * elt_bytes<ELT>() / 4;
    const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x;
    int64_t row, b;
    split_index(unit / LANES, nb, row, b);
    const int64_t k = b * 128 + (threadIdx.x % LANES) * N;
    const bool there = row < a.rows && k < a.H;
    uint32_t gate[W], up[W];
#pragma unroll
    for (int j = 0; j < W; ++j) gate[j] = up[j] = 0;
    if (there) {
        const char* p = static_cast<const char*>(a.x) + (row * a.ldx + k) * elt_bytes<ELT>();
        load_words<W>(gate, p);
        load_words<W>(up, p + a.H * elt_bytes<ELT>());
    }
    float v[N];
    gated<ELT, N, QUANT>(gate, up, v);
    uint32_t amax = amax_of<N>(v);
    if constexpr (QUANT) {
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        const uint32_t code = scale_code128(amax);
        if (!there) return;
        if (threadIdx.x % LANES == 0) a.scales[row * nb + b] = (uint8_t)code;
        const float2 inv = both(__uint_as_float(inv_scale128(code)));
        uint32_t o[N / 4];
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
            const float2 lo = mul2(make_float2(v[4 * j], v[4 * j + 1]), inv), hi = mul2(make_float2(v[4 * j + 2], v[4 * j + 3]), inv);
            o[j] = e4m3x2_from_f32(__float_as_uint(lo.y), __float_as_uint(lo.x)) | e4m3x2_from_f32(__float_as_uint(hi.y), __float_as_uint(hi.x)) << 16;
            if (code == 255u) o[j] = 0x7F7F7F7Fu;
        }
        uint8_t* p = a.data + row * a.H + k;
        if constexpr (N == 16) st16(p, o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
    } else {
        if (!there) return;
        char* p = static_cast<char*>(a.out) + (row * a.H + k) * elt_bytes<ELT>();
        const bool nan = amax > 0x7F800000u;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if constexpr (ELT == Elt::BF16) gate[j] = bf16x2_from_f32(v[2 * j + 1], v[2 * j]);
            else gate[j] = __float_as_uint(v[j]);
            if (nan) gate[j] = canonical_word<ELT>(gate[j]);
        }
        if constexpr (W % 8 == 0) {
#pragma unroll
            for (int j = 0; j < W; j += 8) st32(p + 4 * j, *reinterpret_cast<const uint32_t(*)[8]>(gate + j));
        } else {
            st16(p, gate[0], gate[1], gate[2], gate[3]);
        }
    }
}

// Tiles of 128 rows x C TX columns a block, C columns of R rows a thread, in
// registers between the maximum and the rounding: each element is read once.
// bf16: few columns of many rows, since each column's maximum costs shuffles
// and its scale unpacking, and 64 registers: 16379 x 4096 51.9 us, 6.5 TB/s
// (eight columns of four rows 63 to 73, seven blocks a multiprocessor 54.6, 16
// threads a row 54.6).  fp32: wide loads count for more, 8191 x 4096 48.8 us, 6.2
// TB/s (four columns of eight rows 57 to 66; five or seven blocks a multiprocessor 56.6
// and 51.2).
template <Elt ELT>
struct GateTile {
    static constexpr bool kBf16 = ELT == Elt::BF16;
    static constexpr int kC = kBf16 ? 4 : 8, kX = kBf16 ? 8 : 4, kRows = kBf16 ? 8 : 4, kBlocks = kBf16 ? 8 : 6;
    static constexpr int kThreads = kX * 128 / kRows;
};
template <Elt ELT>
__global__ void __launch_bounds__(GateTile<ELT>::kThreads, GateTile<ELT>::kBlocks) gate_columns_tile_kernel(GateArgs a) {
    let_next_start();
    wait_for_stream();
    constexpr int TX = GateTile<ELT>::kX, R = GateTile<ELT>::kRows, C = GateTile<ELT>::kC, TY = 128 / R, WARPS = TX * TY / 32, W = C * (int)elt_bytes<ELT>() / 4;
    __shared__ __align__(16) uint32_t top[WARPS][C * TX];
    __shared__ __align__(8) uint8_t codes[C * TX];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int64_t c = ((int64_t)blockIdx.x * TX + tx) * C, r0 = (int64_t)blockIdx.y * 128 + ty;
    uint32_t gate[R][W], up[R][W];
    const char* p = static_cast<const char*>(a.x) + (r0 * a.ldx + c) * elt_bytes<ELT>();
#pragma unroll
    for (int i = 0; i < R; ++i, p += TY * a.ldx * elt_bytes<ELT>()) {
#pragma unroll
        for (int j = 0; j < W; ++j) gate[i][j] = up[i][j] = 0;
        if (r0 + TY * i < a.rows && c < a.H) {
            load_words<W>(gate[i], p);
            load_words<W>(up[i], p + a.H * elt_bytes<ELT>());
        }
    }
    float v[R][C];
    uint32_t m[C];
#pragma unroll
    for (int i = 0; i < R; ++i) gated<ELT, C, true>(gate[i], up[i], v[i]);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < R; i += 2) t = absmax3(t, v[i][j], v[i + 1][j]);
        m[j] = __float_as_uint(t) & 0x7FFFFFFFu;
#pragma unroll
        for (int d = TX; d < 32; d *= 2) m[j] = max(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], d));
    }
    if ((threadIdx.x & 31) < TX)
#pragma unroll
        for (int j = 0; j < C; j += 4) *reinterpret_cast<uint4*>(&top[threadIdx.x / 32][C * tx + j]) = make_uint4(m[j], m[j + 1], m[j + 2], m[j + 3]);
    __syncthreads();
    if (threadIdx.x < C * TX) {
        uint32_t amax = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) amax = max(amax, top[w][threadIdx.x]);
        const uint8_t own = (uint8_t)scale_code128(amax);
        codes[threadIdx.x] = own;
        const int64_t column = (int64_t)blockIdx.x * (C * TX) + threadIdx.x;
        if (column < a.H) a.scales[(int64_t)blockIdx.y * a.H + column] = own;
    }
    __syncthreads();
    if (c >= a.H) return;
    float2 inv[C / 2];
    uint32_t nan[C / 4] = {};  // bytes of poisoned columns
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t code = *reinterpret_cast<const uint32_t*>(codes + C * tx + j / 4 * 4) >> (8 * (j & 3)) & 0xFFu;
        (j & 1 ? inv[j / 2].y : inv[j / 2].x) = __uint_as_float(inv_scale128(code));
        nan[j / 4] |= code == 255u ? 0xFFu << (8 * (j & 3)) : 0u;
    }
    uint8_t* to = a.data + r0 * a.H + c;
#pragma unroll
    for (int i = 0; i < R; ++i, to += TY * a.H) {
        if (r0 + TY * i >= a.rows) break;
        uint32_t o[C / 4];
#pragma unroll
        for (int h = 0; h < C / 4; ++h) {
            const float2 lo = mul2(make_float2(v[i][4 * h], v[i][4 * h + 1]), inv[2 * h]),
                         hi = mul2(make_float2(v[i][4 * h + 2], v[i][4 * h + 3]), inv[2 * h + 1]);
            const uint32_t w = e4m3x2_from_f32(__float_as_uint(lo.y), __float_as_uint(lo.x)) |
                               e4m3x2_from_f32(__float_as_uint(hi.y), __float_as_uint(hi.x)) << 16;
            o[h] = lop_select(0x7F7F7F7Fu, w, nan[h]);
        }
        if constexpr (C == 8) *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[C / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(to) = o[0];
    }
}

// Gradients of two gates and their other factors, for the gradients g of a:
// d_up = g silu(x), d_gate = g up silu'(x), silu'(x) = s (1 + x (1 - s)) with s = 1 / (1
// + exp(-x)).  All of s and silu' is there without the scale, which goes into the
// products last.  g up may be out of range where d_gate is not: silu' goes with the
// larger of the two, and of the scale and the smaller one that comes first which
// takes the product towards 1.
template <Elt ELT>
struct GateGrad {
    float2 gate, up;
    __device__ __forceinline__ GateGrad(float2 g, float2 x, float2 u) {
        const Scaled c(x);
        const float2 e = exp_scaled<ELT, true>(x, c), d = fma2(e, both(1.0f), c.scale), inv = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        const float2 slope = mul2(inv, fma2(x, mul2(e, inv), both(1.0f)));
        up = mul2(mul2(g, mul2(x, inv)), c.scale);
        gate = make_float2(product(g.x, u.x, slope.x, c.scale.x), product(g.y, u.y, slope.y, c.scale.y));
    }
    __device__ __forceinline__ static float product(float g, float u, float slope, float scale) {
        const bool first = fabsf(g) > fabsf(u);
        const float least = first ? u : g, most = fmul(first ? g : u, slope);
        const bool high = fabsf(most) >= 1.0f;
        return fmul(fmul(most, high ? scale : least), high ? least : scale);
    }
};

// Any alignment and any H, every form but COLUMNS: one row to blockIdx.x, its
// 1x128 blocks to the warps of blockIdx.y in turn, an element at a time,
// neighbours to neighbouring lanes.  Bound by instructions: 8191 x 4095 bf16 to FP8
// 44.1 us, its gradient 67.4 (four or six blocks a multiprocessor 73 and 68), 3.8 and 5.0 TB/s.
template <Elt ELT, GateForm FORM>
__global__ void __launch_bounds__(256, FORM == GateForm::GRAD ? 5 : 0) gate_any_kernel(GateArgs a, int nb) {
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31, H = (int)a.H;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* x = static_cast<const char*>(a.x) + row * a.ldx * elt_bytes<ELT>();
        const char* u = x + a.H * elt_bytes<ELT>();
        const char* g = FORM == GateForm::GRAD ? static_cast<const char*>(a.g) + row * a.ldg * elt_bytes<ELT>() : nullptr;
        for (int b = blockIdx.y * 8 + threadIdx.x / 32; b < nb; b += gridDim.y * 8) {
            const int k = b * 128 + lane;
            uint32_t gate[4], up[4], of[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool there = k + 32 * q < H;
                gate[q] = there ? load_f32<ELT>(x, k + 32 * q) : 0u;
                up[q] = there ? load_f32<ELT>(u, k + 32 * q) : 0u;
                of[q] = FORM == GateForm::GRAD && there ? load_f32<ELT>(g, k + 32 * q) : 0u;
            }
            if constexpr (FORM == GateForm::GRAD) {
                char* to = static_cast<char*>(a.out) + row * 2 * a.H * elt_bytes<ELT>();
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const auto two = [q](const uint32_t(&w)[4]) { return make_float2(__uint_as_float(w[q]), __uint_as_float(w[q + 1])); };
                    const GateGrad<ELT> d(two(of), two(gate), two(up));
                    if (k + 32 * q < H) {
                        store_f32<ELT>(to, k + 32 * q, d.gate.x);
                        store_f32<ELT>(to, H + (int64_t)k + 32 * q, d.up.x);
                    }
                    if (k + 32 * q + 32 < H) {
                        store_f32<ELT>(to, k + 32 * q + 32, d.gate.y);
                        store_f32<ELT>(to, H + (int64_t)k + 32 * q + 32, d.up.y);
                    }
                }
            } else {
                constexpr bool QUANT = FORM == GateForm::ROWS;
                float v[4];
                gated_loose<ELT, 4, QUANT>(gate, up, v);
                if constexpr (QUANT) {
                    const uint32_t code = scale_code128(__reduce_max_sync(0xFFFFFFFFu, amax_of<4>(v)));
                    if (lane == 0) a.scales[row * nb + b] = (uint8_t)code;
                    const float2 inv = both(__uint_as_float(inv_scale128(code)));
                    uint8_t* to = a.data + row * a.H;
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const float2 p = mul2(make_float2(v[q], v[q + 1]), inv);
                        const uint32_t two = code == 255u ? 0x7F7Fu : e4m3x2_from_f32(__float_as_uint(p.y), __float_as_uint(p.x));
                        if (k + 32 * q < H) to[k + 32 * q] = (uint8_t)two;
                        if (k + 32 * q + 32 < H) to[k + 32 * q + 32] = (uint8_t)(two >> 8);
                    }
                } else {
                    char* to = static_cast<char*>(a.out) + row * a.H * elt_bytes<ELT>();
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (k + 32 * q < H) store_f32<ELT>(to, k + 32 * q, v[q]);
                }
            }
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
    uint32_t gate[R], up[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + Y * i;
        const bool there = r < a.rows && c < a.H;
        gate[i] = there ? load_f32<ELT>(a.x, r * a.ldx + c) : 0u;
        up[i] = there ? load_f32<ELT>(a.x, r * a.ldx + a.H + c) : 0u;
    }
    float v[R];
    gated_loose<ELT, R, true>(gate, up, v);
    uint32_t amax = amax_of<R>(v);
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

// A unit of 16 elements of both halves a thread.  Bound by HBM: 8191 x 7184 bf16
// 85.3 us, 6.9 TB/s (four or six blocks a multiprocessor 87 and 103).
template <Elt ELT>
__global__ void __launch_bounds__(256, ELT == Elt::BF16 ? 5 : 4) gate_grad_kernel(GateArgs a, int64_t nu) {
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
        const GateGrad<ELT> d(g.f2(j), gate.f2(j), up.f2(j));
        gate.set2(j, d.gate.x, d.gate.y);
        up.set2(j, d.up.x, d.up.y);
        top = max(max(top, __float_as_uint(d.gate.x) & 0x7FFFFFFFu), __float_as_uint(d.gate.y) & 0x7FFFFFFFu);
        top = max(max(top, __float_as_uint(d.up.x) & 0x7FFFFFFFu), __float_as_uint(d.up.y) & 0x7FFFFFFFu);
    }
    if (top > 0x7F800000u) gate.canonical(), up.canonical();
    gate.store(a.out, row * 2 * a.H + k);
    up.store(a.out, row * 2 * a.H + a.H + k);
}

constexpr int64_t kMostBlocks = INT64_C(0x7FFFFFFF);

template <Elt ELT, GateForm FORM>
cudaError_t any_launch(const GateArgs& a, cudaStream_t s) {
    // few rows are cut into slices so that the device is full
    const int64_t nb = ceil_div(a.H, 128), slices = ceil_div(nb, 8), wanted = ceil_div((int64_t)sm_count() * 8, a.rows);
    const dim3 grid((unsigned)(a.rows < kMostBlocks ? a.rows : kMostBlocks),
                    (unsigned)(wanted < 1 ? 1 : wanted < slices ? wanted : slices < 65535 ? slices : 65535));
    return launch_overlapped(gate_any_kernel<ELT, FORM>, grid, 256, 0, 0, s, a, (int)nb);
}

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
        return any_launch<ELT, GateForm::GRAD>(a, s);
    }
    if (form == GateForm::COLUMNS) {
        using Tile = GateTile<ELT>;
        constexpr int64_t bytes = Tile::kC * elt_bytes<ELT>();  // of a thread's columns
        const bool tiled = a.H % Tile::kC == 0 && on_bytes(a.x, bytes) && (a.rows <= 1 || a.ldx % Tile::kC == 0) && on_bytes(a.data, Tile::kC);
        // blockIdx.y reaches 65535: 2^23 rows at a time
        for (int64_t r0 = 0; r0 < a.rows; r0 += INT64_C(128) * 65535) {
            GateArgs p = a;
            p.rows = a.rows - r0 < INT64_C(128) * 65535 ? a.rows - r0 : INT64_C(128) * 65535;
            p.x = static_cast<const char*>(a.x) + r0 * a.ldx * elt_bytes<ELT>();
            p.data = a.data + r0 * a.H;
            p.scales = a.scales + r0 / 128 * a.H;
            const unsigned y = (unsigned)ceil_div(p.rows, 128);
            const cudaError_t e =
                tiled ? launch_overlapped(gate_columns_tile_kernel<ELT>, dim3((unsigned)ceil_div(a.H, Tile::kC * Tile::kX), y), Tile::kThreads, 0, 0, s, p)
                      : launch_overlapped(gate_columns_kernel<ELT>, dim3((unsigned)ceil_div(a.H, 64), y), 512, 0, 0, s, p);
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
    return quant ? any_launch<ELT, GateForm::ROWS>(a, s) : any_launch<ELT, GateForm::PLAIN>(a, s);
}

}  // namespace

cudaError_t launch_gate(Elt elt, GateForm form, const GateArgs& a, cudaStream_t s) {
    const cudaError_t e = elt == Elt::BF16 ? launch<Elt::BF16>(form, a, s) : launch<Elt::FP32>(form, a, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace mxq
