// mxq_route.cu -- a router's logits to experts and weights, and the gradient.
//
//   s = softmax(l) or 1 / (1 + exp(-l))       c = s + bias
//   a group's score: the sum of the group_top largest c of its experts
//   chosen: the topk largest c of the topk_groups best groups, ties to the
//   lowest index;   w_j = scale s_j, or scale s_j / (sum of the chosen s)
//
// Which expert is ahead is what exact arithmetic says.  Without a bias, and
// with groups scored by their largest expert, the logits' own order is that of
// the scores.  Otherwise c is computed in fp32, and a token for which two
// neighbours of the order lie nearer than the error of that is decided again
// in 64 bits (a few of a thousand tokens).
//
// A warp to a token, VPL consecutive experts to a lane, in registers.
#include "mxq_device.cuh"
#include "mxq_e4m3.cuh"
#include "mxq_layer.h"
#include "mxq_launch.cuh"

namespace mxq {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 4;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int d = 16; d; d /= 2) v = fadd(v, __shfl_xor_sync(kAll, v, d));
    return v;
}

// Numbers as keys of the same order: a larger number has a larger key, -0 that
// of 0, -inf the least one, above 0, which stands for "not to be chosen".
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(fadd(v, 0.0f));
    return u ^ ((int32_t)u < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
    return u ^ ((int64_t)u < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double of_key(uint64_t k) {
    return __longlong_as_double((long long)(k ^ ((int64_t)k < 0 ? 1ull << 63 : ~0ull)));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = warp_max((uint32_t)(k >> 32));
    const uint32_t lo = warp_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ float warp_max(float v) {
    asm volatile("redux.sync.max.f32 %0, %0, 0xFFFFFFFF;" : "+f"(v));
    return v;
}
__device__ __forceinline__ double warp_max(double v) { return of_key(warp_max(key_of(v))); }

// The two largest of some numbers.
template <typename Real>
struct Top2 {
    Real a = (Real)-kInf, b = (Real)-kInf;
    __device__ __forceinline__ void add(Real v) {
        b = max(b, min(a, v));
        a = max(a, v);
    }
    __device__ __forceinline__ void add(const Top2& o) {
        b = max(max(b, o.b), min(a, o.a));
        a = max(a, o.a);
    }
    __device__ __forceinline__ void merge(int d) {
        Top2 o;
        o.a = __shfl_xor_sync(kAll, a, d);
        o.b = __shfl_xor_sync(kAll, b, d);
        add(o);
    }
    // The group's score; -inf where no expert of it can be chosen.
    __device__ __forceinline__ Real score(int top) const { return top == 1 || b == (Real)-kInf ? a : a + b; }
    __device__ __forceinline__ Real size() const {
        return (a == (Real)-kInf ? (Real)0 : fabs(a)) + (b == (Real)-kInf ? (Real)0 : fabs(b));
    }
};
template <int N, typename Real>
__device__ __forceinline__ Top2<Real> top2_of(const Real* c) {
    Top2<Real> t;
    if constexpr (N == 1) {
        t.a = c[0];
    } else {
        t = top2_of<N / 2>(c);
        t.add(top2_of<N / 2>(c + N / 2));
    }
    return t;
}

template <Elt ELT>
__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
    return __uint_as_float(load_f32<ELT>(a.logits, t * a.ld + e));
}

// VPL consecutive logits, -inf behind the last expert.
template <Elt ELT, int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float (&x)[VPL]) {
    constexpr int kWords = VPL * (ELT == Elt::BF16 ? 2 : 4) / 16;  // 16-byte words of a lane
    if (kWords > 0 && a.vector) {
        if (lane * VPL < a.E) {
            uint32_t w[kWords ? 4 * kWords : 1];
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(a.logits) + (t * a.ld + lane * VPL) * elt_bytes<ELT>());
#pragma unroll
            for (int q = 0; q < kWords; ++q) {
                const uint4 v = __ldg(p + q);
                w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                x[i] = __uint_as_float(ELT == Elt::FP32 ? w[kWords ? i : 0] : i & 1 ? w[kWords ? i / 2 : 0] & 0xFFFF0000u : w[kWords ? i / 2 : 0] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) x[i] = -kInf;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) x[i] = lane * VPL + i < a.E ? logit<ELT>(a, t, lane * VPL + i) : -kInf;
    }
}

// How the experts' groups lie: none, a power of two of whole lanes each, or otherwise.
enum Groups { NONE, LANES, ANY };

// Takes the experts of all but the best groups out (c = -inf).
template <int VPL, Groups GROUPS, typename Real>
__device__ __forceinline__ void best_groups(const RouteArgs& a, int lane, Real (&c)[VPL], Real err, bool& unsure) {
    constexpr Real kRound = (Real)(1.0 / (1 << 22));
    Top2<Real> top;
    int group = lane, shift = 0, ahead = 0;
    if constexpr (GROUPS == LANES) {
        shift = a.group_shift;
        group = lane >> shift;
        top = top2_of<VPL>(c);
        for (int d = 1; d < 1 << shift; d *= 2) top.merge(d);
    } else {
        for (int g = 0; g < a.groups; ++g) {
            Top2<Real> of;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (lane * VPL + i >= g * a.group_size && lane * VPL + i < (g + 1) * a.group_size) of.add(c[i]);
            for (int d = 1; d < 32; d *= 2) of.merge(d);
            if (lane == g) top = of;
        }
    }
    const Real mine = top.score(a.group_top);
    // a group's lanes share the comparisons with the others
    for (int g0 = 0; g0 < a.groups; g0 += 1 << shift) {
        const int g = g0 + (lane & ((1 << shift) - 1));
        const Real other = __shfl_sync(kAll, mine, (g << shift) & 31);
        ahead += g < a.groups && (other > mine || (other == mine && g < group)) ? 1 : 0;
    }
    for (int d = 1; d < 1 << shift; d *= 2) ahead += __shfl_xor_sync(kAll, ahead, d);
    const bool real = group < a.groups, kept = real && ahead < a.topk_groups;
    if (err >= (Real)0 && a.topk_groups < a.groups) {
        const Real least = -warp_max(kept ? -mine : (Real)-kInf), next = warp_max(real && !kept ? mine : (Real)-kInf);
        const Real tol = 2 * a.group_top * err + kRound * warp_max(top.size());
        if (next > (Real)-kInf && least - next <= tol) unsure = true;
    }
    if constexpr (GROUPS == LANES) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = kept ? c[i] : (Real)-kInf;
    } else {
        const unsigned mask = __ballot_sync(kAll, kept);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane * VPL + i >= a.E || !(mask >> ((lane * VPL + i) / a.group_size) & 1)) c[i] = (Real)-kInf;
    }
}

// Can two neighbours of the order, last in front of e, not be told apart?
// Equal logits with equal biases are ties, which the index decides.
template <Elt ELT, typename Real>
__device__ __forceinline__ bool too_near(const RouteArgs& a, int64_t t, Real err, Real last_c, int last, Real c, int e) {
    constexpr Real kRound = (Real)(1.0 / (1 << 22));
    return last_c - c <= 2 * err + kRound * max(fabs(last_c), fabs(c)) &&
           !(logit<ELT>(a, t, last) == logit<ELT>(a, t, e) && (!a.bias || a.bias[last] == a.bias[e]));
}

// The topk largest of c, one after the other: lane j's result is the j-th, -1
// for none.  c is -inf for what cannot be chosen.  err: how far a c may be
// off what exact arithmetic gives, besides its last rounding; neighbours that
// cannot be told apart set `unsure`.  A negative err: c is taken as it is.
template <Elt ELT, int VPL, typename Real>
__device__ __forceinline__ int choose_in_turn(const RouteArgs& a, int64_t t, int lane, const Real (&c)[VPL], Real err, bool& unsure) {
    using Key = decltype(key_of(Real()));
    Key key[VPL], top = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = c[i] > (Real)-kInf ? key_of(c[i]) : (Key)0;
        top = max(top, key[i]);
    }
    int id = -1, last = -1;
    Real last_c = 0;
    const int rounds = a.topk + (err >= (Real)0 ? 1 : 0);
    for (int j = 0; j < rounds; ++j) {
        const Key best = warp_max(top);
        if (best == 0) break;
        const int src = __ffs(__ballot_sync(kAll, top == best)) - 1;
        int e = 0;
        if (lane == src) {
            bool found = false;
            top = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (!found && key[i] == best) {
                    found = true;
                    e = lane * VPL + i;
                    key[i] = 0;
                }
                top = max(top, key[i]);
            }
        }
        e = __shfl_sync(kAll, e, src);
        if (j < a.topk && lane == j) id = e;
        if (err >= (Real)0) {
            const Real now = of_key(best);
            if (j && too_near<ELT>(a, t, err, last_c, last, now, e)) unsure = true;
            last = e;
            last_c = now;
        }
    }
    return id;
}

// The same for fp32 in fewer steps.  The topk + 1 largest are among the values
// that reach the (topk + 1)-th largest of the lanes' own largest ones: a dozen
// for topk 8.  Those go to shared memory, one to a lane, and each counts how
// many are ahead of it.  More than 32 of them are chosen in turn.
template <Elt ELT, int VPL>
__device__ __forceinline__ int choose32(const RouteArgs& a, int64_t t, int lane, const float (&c)[VPL], float err, bool& unsure, uint64_t* list) {
    float left = c[0], from = -kInf;
#pragma unroll
    for (int i = 1; i < VPL; ++i) left = max(left, c[i]);
    const int rounds = a.topk + (err >= 0.0f ? 1 : 0);
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        from = warp_max(left);
        left = left == from ? -kInf : left;
    }
    from = max(from, -3.4028235e38f);  // with fewer lanes than rounds, all that can be chosen
    int mine = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) mine += c[i] >= from ? 1 : 0;
    int at = 0, n = 0;
#pragma unroll
    for (int b = 0; (1 << b) <= VPL; ++b) {
        const unsigned bit = __ballot_sync(kAll, mine >> b & 1);
        at += __popc(bit & ((1u << lane) - 1)) << b;
        n += __popc(bit) << b;
    }
    if (n > 32) return choose_in_turn<ELT, VPL, float>(a, t, lane, c, err, unsure);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (c[i] >= from) list[at++] = (uint64_t)__float_as_uint(c[i]) << 32 | (uint32_t)(lane * VPL + i);
    __syncwarp();
    uint64_t own = 0;
    if (lane < n) {  // the order of the keys: by value, then the lower index first
        own = list[lane];
        own = (uint64_t)key_of(__uint_as_float((uint32_t)(own >> 32))) << 32 | (uint32_t)~(uint32_t)own;
    }
    list[lane] = own;
    __syncwarp();
    int rank = 0;
#pragma unroll 2
    for (int j = 0; j < n; j += 2) {  // behind the last there are zeros
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(list + j);
        rank += k.x > own ? 1 : 0;
        rank += k.y > own ? 1 : 0;
    }
    __syncwarp();
    if (lane < n) list[rank] = own;
    __syncwarp();
    int id = -1;
    if (lane < a.topk && lane < n) {
        const uint64_t k = list[lane];
        id = (int)~(uint32_t)k;
        if (err >= 0.0f && lane + 1 < n) {
            const uint64_t l = list[lane + 1];
            unsure |= too_near<ELT>(a, t, err, of_key((uint32_t)(k >> 32)), id, of_key((uint32_t)(l >> 32)), (int)~(uint32_t)l);
        }
    }
    return id;
}

// The largest; NaN if one is.
template <int N>
__device__ __forceinline__ float max_nan(const float (&v)[N]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; i += 2) asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[i]), "f"(v[i + 1 < N ? i + 1 : i]));
    return m;
}

template <int VPL>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int lane, float (&b)[VPL]) {
    if (VPL % 4 == 0 && a.vector) {
        if (lane * VPL < a.E) {
            const float4* p = reinterpret_cast<const float4*>(a.bias + lane * VPL);
#pragma unroll
            for (int q = 0; q < VPL / 4; ++q) {
                const float4 v = __ldg(p + q);
                b[4 * q] = v.x, b[4 * q + 1] = v.y, b[4 * q + 2] = v.z, b[4 * q + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane * VPL + i < a.E) b[i] = __ldg(a.bias + lane * VPL + i);
    }
}

// Scores of VPL logits: 1 / (1 + exp(-x)), or exp(x - m) for the softmax; 0 for -inf.
template <int VPL>
__device__ __forceinline__ void scores(const RouteArgs& a, const float (&x)[VPL], float m, float (&s)[VPL]) {
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; i += 2) {
            const int j = VPL > 1 ? i + 1 : i;
            const float2 e = exp_neg2(make_float2(min_nan(fabsf(x[i]), kExpEnd), min_nan(fabsf(x[j]), kExpEnd)));
            const float2 inv = make_float2(rcp_approx(fadd(1.0f, e.x)), rcp_approx(fadd(1.0f, e.y))), low = mul2(e, inv);
            s[i] = x[i] < 0.0f ? low.x : inv.x;
            s[j] = x[j] < 0.0f ? low.y : inv.y;
        }
    } else {
        const float from = m == -kInf ? 0.0f : m;  // a row of -inf alone
#pragma unroll
        for (int i = 0; i < VPL; i += 2) {
            const int j = VPL > 1 ? i + 1 : i;
            const float2 e = exp_neg2(make_float2(min_nan(from - x[i], kExpEnd), min_nan(from - x[j], kExpEnd)));
            s[i] = e.x;
            s[j] = e.y;
        }
    }
}

// The same in 64 bits.
template <Elt ELT, int VPL, Groups GROUPS>
__device__ __noinline__ int choose64(const RouteArgs& a, int64_t t, int lane) {
    float x[VPL];
    load_logits<ELT, VPL>(a, t, lane, x);
    float m = -kInf;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = max(m, x[i]);
    m = warp_max(m);
    double c[VPL], sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < VPL; ++i) {
        c[i] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : exp((double)x[i] - (double)m);
        sum += c[i];
    }
    for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(kAll, sum, d);
#pragma unroll 1
    for (int i = 0; i < VPL; ++i) {
        if (!a.sigmoid) c[i] /= sum;
        if (a.bias && lane * VPL + i < a.E) c[i] += (double)a.bias[lane * VPL + i];
        if (x[i] == -kInf) c[i] = -(double)kInf;
    }
    bool unsure = false;
    if constexpr (GROUPS != NONE) best_groups<VPL, GROUPS, double>(a, lane, c, -1.0, unsure);
    return choose_in_turn<ELT, VPL, double>(a, t, lane, c, -1.0, unsure);
}

// The chosen experts' scores up to a common factor of the row, lane j for
// choice j (0 for none), and their sum.  The factor keeps a row whose scores
// all underflow from being 0 / 0: softmax scores are taken relative to the
// largest chosen one, sigmoid's are multiplied by exp(-m) for a largest logit m < 0.
struct Chosen {
    float u, sum, rest;  // rest: 1 - sigmoid
    __device__ __forceinline__ Chosen(float x, bool sigmoid) {
        const float m = warp_max(x);
        rest = 1.0f;
        if (x == -kInf) {
            u = 0.0f;
        } else if (!sigmoid) {
            u = exp_neg(m - x);
        } else {
            const Sigmoid s(x);
            rest = s.rest;
            u = x > 0.0f ? s.s : fmul(exp_neg(min(m, 0.0f) - x), s.rest);
        }
        sum = lane_sum(u);
    }
};

template <Elt ELT, int VPL, Groups GROUPS>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ __align__(16) uint64_t lists[kWarps][32];
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.T) return;
    float c[VPL];
    load_logits<ELT, VPL>(a, t, lane, c);
    float m = max_nan<VPL>(c);
    bool bad = m != m;
    if (!a.sigmoid) {
        m = warp_max(m);
        bad |= m == kInf;
    }
    float total = 0.0f, err = -1.0f;
    const bool scored = a.bias || (GROUPS != NONE && a.group_top > 1);
    if (scored || !(a.sigmoid || a.renorm)) {
        float s[VPL];
        scores<VPL>(a, c, m, s);
        if (!a.sigmoid) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) total = fadd(total, s[i]);
            total = lane_sum(total);
        }
        if (scored) {
            // in units of 2^-24 of the largest score: two of exp_neg and the sum, or the reciprocal, and a sum's VPL + 5 terms
            const float most = a.sigmoid ? 1.0f : fdiv(1.0f, total);
            err = (a.sigmoid ? 10.0f : VPL + 20.0f) * 5.9604645e-8f * most;
            float b[VPL];
#pragma unroll
            for (int i = 0; i < VPL; ++i) b[i] = 0.0f;
            if (a.bias) {
                load_bias<VPL>(a, lane, b);
                const float top = max_nan<VPL>(b);
                bad |= top != top;
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float v = fadd(a.sigmoid ? s[i] : fmul(s[i], most), b[i]);
                c[i] = c[i] > -kInf ? v : c[i];
            }
        }
    }
    bad = __any_sync(kAll, bad);
    int id = lane;  // a row that cannot be scored: valid experts, and NaN as their weights
    float x = -kInf;
    if (!bad) {
        bool unsure = false;
        if constexpr (GROUPS != NONE) best_groups<VPL, GROUPS, float>(a, lane, c, err, unsure);
        id = choose32<ELT, VPL>(a, t, lane, c, err, unsure, lists[threadIdx.x / 32]);
        if (__any_sync(kAll, unsure)) id = choose64<ELT, VPL, GROUPS>(a, t, lane);
        if (id >= 0) x = logit<ELT>(a, t, id);
    }
    float w = x == -kInf ? 0.0f : a.sigmoid ? Sigmoid(x).s : exp_neg(m - x);
    if (a.renorm) {
        float sum = lane_sum(w);
        if (sum < 1e-3f) {  // the chosen scores are small, or underflow
            const Chosen chosen(x, a.sigmoid);
            w = chosen.u;
            sum = chosen.sum;
        }
        w = sum > 0.0f ? fdiv(w, sum) : 0.0f;
    } else if (!a.sigmoid) {
        w = total > 0.0f ? fdiv(w, total) : 0.0f;
    }
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = id;
        a.weights[t * a.topk + lane] = bad ? __uint_as_float(0x7FC00000u) : fmul(a.scale, w);
    }
}

// d_logits for the gradient g of the weights.  With u_j = s_j / (sum of the
// chosen s): renormalised, d_j = scale u_j (g_j - sum_i g_i u_i), for sigmoid
// times 1 - s_j, and zero for what was not chosen (the softmax's sum cancels);
// else d_e = scale (s_e g_e [chosen] - s_e sum_j g_j s_j) for softmax and scale
// g_j s_j (1 - s_j) for sigmoid.  A warp to a token.
template <Elt ELT, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ __align__(16) float rows[kWarps][32 * VPL];
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.T) return;
    int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
    if (id >= a.E) id = -1;
    const float g = id >= 0 ? fmul(a.scale, a.g[t * a.topk + lane]) : 0.0f;
    const float x = id >= 0 ? logit<ELT>(a, t, id) : -kInf;
    float d[VPL], v;
    if (a.sigmoid || a.renorm) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
        const Chosen chosen(x, a.sigmoid);
        if (a.renorm) {
            const float u = id >= 0 ? fdiv(chosen.u, chosen.sum) : 0.0f;
            v = fmul(u, fadd(g, -lane_sum(fmul(g, u))));
            if (a.sigmoid) v = fmul(v, chosen.rest);
        } else {
            const Sigmoid s(x);
            v = fmul(g, fmul(s.s, s.rest));
        }
        if (id < 0 || x == -kInf) v = 0.0f;
    } else {
        load_logits<ELT, VPL>(a, t, lane, d);
        float m = max_nan<VPL>(d);
        m = __any_sync(kAll, m != m) ? __uint_as_float(0x7FC00000u) : warp_max(m);
        float total = 0.0f;
        scores<VPL>(a, d, m, d);
#pragma unroll
        for (int i = 0; i < VPL; ++i) total = fadd(total, d[i]);
        total = lane_sum(total);
        const float inv = total == 0.0f ? 0.0f : fdiv(1.0f, total);
        v = x == -kInf ? 0.0f : fmul(g, fmul(exp_neg(m - x), inv));
        const float all = -fmul(inv, lane_sum(v));
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = fmul(d[i], all);
    }
    float* row = rows[threadIdx.x / 32];
    // a choice that is its token's only one of an expert adds to what the others leave; of several of one expert the first adds
    // all, in their order
    if (id >= 0) row[id] = __uint_as_float(lane);
    __syncwarp();
    bool first = id >= 0;
    if (__any_sync(kAll, first && __float_as_uint(row[id]) != lane)) {
        float sum = 0.0f;
        for (int j = 0; j < a.topk; ++j) {
            const int e = __shfl_sync(kAll, id, j);
            const float add = __shfl_sync(kAll, v, j);
            if (e == id) {
                sum = fadd(sum, add);
                first &= j >= lane;
            }
        }
        v = sum;
    }
    __syncwarp();
    if constexpr (VPL % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) *reinterpret_cast<float4*>(row + lane * VPL + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) row[lane * VPL + i] = d[i];
    }
    __syncwarp();
    if (first) row[id] = fadd(row[id], v);
    __syncwarp();
    constexpr int kPer = ELT == Elt::BF16 ? 8 : 4;  // 16 bytes
    // NaN comes out canonical: only a row with a NaN or an infinity can have one
    const bool odd = __any_sync(kAll, !(fabsf(v) < kInf) || !(fabsf(d[0]) < kInf));
    if (a.vector && !odd) {
        for (int e = lane * kPer; e < a.E; e += 32 * kPer) {
            const float4 p = *reinterpret_cast<const float4*>(row + e);
            uint4 w;
            if constexpr (ELT == Elt::BF16) {
                const float4 q = *reinterpret_cast<const float4*>(row + e + 4);
                w = make_uint4(bf16x2_from_f32(p.y, p.x), bf16x2_from_f32(p.w, p.z), bf16x2_from_f32(q.y, q.x), bf16x2_from_f32(q.w, q.z));
            } else {
                w = make_uint4(__float_as_uint(p.x), __float_as_uint(p.y), __float_as_uint(p.z), __float_as_uint(p.w));
            }
            *reinterpret_cast<uint4*>(static_cast<char*>(a.d_logits) + (t * a.E + e) * elt_bytes<ELT>()) = w;
        }
    } else {
        for (int e = lane; e < a.E; e += 32) store_f32<ELT>(a.d_logits, t * a.E + e, row[e]);
    }
}

template <Elt ELT, int VPL>
cudaError_t launch(bool grad, RouteArgs a, cudaStream_t s) {
    // whole lanes of 16-byte words in, and out for the gradient
    a.vector = a.E % VPL == 0 && on_bytes(a.logits, 16) && (a.T <= 1 || a.ld * elt_bytes<ELT>() % 16 == 0) && on_bytes(a.bias, 16) &&
               (!grad || (a.E * elt_bytes<ELT>() % 16 == 0 && on_bytes(a.d_logits, 16)));
    const dim3 grid((unsigned)ceil_div(a.T, kWarps));
    if (grad) return launch_overlapped(route_grad_kernel<ELT, VPL>, grid, kWarps * 32, 0, 0, s, a);
    if (a.groups == 1) return launch_overlapped(route_kernel<ELT, VPL, NONE>, grid, kWarps * 32, 0, 0, s, a);
    a.group_size = a.E / a.groups;
    for (int shift = 0; shift < 6; ++shift)
        if (VPL << shift == a.group_size) {
            a.group_shift = shift;
            return launch_overlapped(route_kernel<ELT, VPL, LANES>, grid, kWarps * 32, 0, 0, s, a);
        }
    return launch_overlapped(route_kernel<ELT, VPL, ANY>, grid, kWarps * 32, 0, 0, s, a);
}

template <Elt ELT>
cudaError_t launch(bool grad, const RouteArgs& a, cudaStream_t s) {
    if (a.E <= 32) return launch<ELT, 1>(grad, a, s);
    if (a.E <= 64) return launch<ELT, 2>(grad, a, s);
    if (a.E <= 128) return launch<ELT, 4>(grad, a, s);
    if (a.E <= 256) return launch<ELT, 8>(grad, a, s);
    if (a.E <= 512) return launch<ELT, 16>(grad, a, s);
    return launch<ELT, 32>(grad, a, s);
}

}  // namespace

cudaError_t launch_route(Elt elt, bool grad, const RouteArgs& a, cudaStream_t s) {
    const cudaError_t e = elt == Elt::BF16 ? launch<Elt::BF16>(grad, a, s) : launch<Elt::FP32>(grad, a, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace mxq
