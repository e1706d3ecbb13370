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

// Numbers as keys of the same order: a larger number has a larger key, -inf
// the least one, above 0, which stands for "not to be chosen".
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((int32_t)u < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((int32_t)k < 0 ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
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
__device__ __forceinline__ float warp_max(float v) { return of_key(warp_max(key_of(v))); }

template <typename Real>
struct Top2 {
    Real a = (Real)-kInf, b = (Real)-kInf;
    __device__ __forceinline__ void add(Real v) {
        b = v > a ? a : v > b ? v : b;
        a = v > a ? v : a;
    }
    __device__ __forceinline__ void merge(int d) {
        const Real oa = __shfl_xor_sync(kAll, a, d), ob = __shfl_xor_sync(kAll, b, d);
        add(oa);
        add(ob);
    }
    // The group's score; -inf where no expert of it can be chosen.
    __device__ __forceinline__ Real score(int top) const { return top == 1 || b == (Real)-kInf ? a : a + b; }
};

template <Elt ELT>
__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
    return fadd(__uint_as_float(load_f32<ELT>(a.logits, t * a.ld + e)), 0.0f);  // -0 becomes 0, which is its equal
}

// VPL consecutive logits, -inf behind the last expert.
template <Elt ELT, int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float (&x)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = lane * VPL + i < a.E ? logit<ELT>(a, t, lane * VPL + i) : -kInf;
}

// The topk largest of c in the best groups: lane j's result is the j-th, -1
// for none.  c is -inf for what cannot be chosen.  err: how far a c may be
// off what exact arithmetic gives; two that cannot be told apart set `unsure`.
// A negative err: c is taken as it is.
template <Elt ELT, int VPL, typename Real>
__device__ __forceinline__ int choose(const RouteArgs& a, int64_t t, int lane, Real (&c)[VPL], Real err, bool& unsure) {
    using Key = decltype(key_of(Real()));
    constexpr Real kRound = (Real)(1.0 / (1 << 22));
    if (a.groups > 1) {
        const int size = a.E / a.groups, lanes = size / VPL;
        // a lane's group and its score; every lane of a group the same
        Real mine = (Real)-kInf;
        int group = lane, step = 1;
        if (lanes * VPL == size && (lanes & (lanes - 1)) == 0) {
            group = lane / lanes, step = lanes;
            Top2<Real> top;
#pragma unroll
            for (int i = 0; i < VPL; ++i) top.add(c[i]);
            for (int d = 1; d < lanes; d *= 2) top.merge(d);
            mine = top.score(a.group_top);
        } else {
            for (int g = 0; g < a.groups; ++g) {
                Top2<Real> top;
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if ((lane * VPL + i) / size == g) top.add(c[i]);
                for (int d = 1; d < 32; d *= 2) top.merge(d);
                if (lane == g) mine = top.score(a.group_top);
            }
        }
        int ahead = 0;
        for (int g = 0; g < a.groups; ++g) {
            const Real other = __shfl_sync(kAll, mine, g * step);
            ahead += other > mine || (other == mine && g < group) ? 1 : 0;
        }
        const bool real = group < a.groups && lane == group * step, kept = real && ahead < a.topk_groups;
        if (err >= (Real)0 && a.topk_groups < a.groups) {
            const Real least = -of_key(warp_max(key_of(kept ? -mine : (Real)-kInf)));
            const Real next = of_key(warp_max(key_of(real && !kept ? mine : (Real)-kInf)));
            const Real tol = 2 * a.group_top * err + kRound * max(fabs(least), fabs(next));
            if (next > (Real)-kInf && least - next <= tol) unsure = true;
        }
        const unsigned mask = __ballot_sync(kAll, kept);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane * VPL + i >= a.E || !(mask >> ((lane * VPL + i) / size * step) & 1)) c[i] = (Real)-kInf;
    }
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
            if (j && last_c - now <= 2 * err + kRound * max(fabs(last_c), fabs(now)) &&
                !(logit<ELT>(a, t, last) == logit<ELT>(a, t, e) && (!a.bias || a.bias[last] == a.bias[e])))
                unsure = true;
            last = e;
            last_c = now;
        }
    }
    return id;
}

// The same in 64 bits.
template <Elt ELT, int VPL>
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
    return choose<ELT, VPL, double>(a, t, lane, c, -1.0, unsure);
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

template <Elt ELT, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.T) return;
    float c[VPL];
    load_logits<ELT, VPL>(a, t, lane, c);
    bool bad = false;
    float m = -kInf;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        bad |= c[i] != c[i];
        m = max(m, c[i]);
    }
    m = warp_max(m);
    bad |= !a.sigmoid && m == kInf;
    float total = 0.0f, err = -1.0f;
    const bool scored = a.bias || (a.groups > 1 && a.group_top > 1);
    if (scored || !(a.sigmoid || a.renorm)) {
        float s[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            s[i] = c[i] == -kInf ? 0.0f : a.sigmoid ? Sigmoid(c[i]).s : exp_neg(m - c[i]);
            total = fadd(total, s[i]);
        }
        total = lane_sum(total);
        if (scored) {
            // in units of 2^-24 of the largest score: two of exp_neg and the sum, or the reciprocal, and a sum's VPL + 5 terms
            const float most = a.sigmoid ? 1.0f : fdiv(1.0f, total);
            constexpr float kStep = 5.9604645e-8f;
            err = (a.sigmoid ? 10.0f : VPL + 20.0f) * kStep * most;
            float size = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float b = a.bias && lane * VPL + i < a.E ? a.bias[lane * VPL + i] : 0.0f;
                bad |= b != b;
                if (c[i] > -kInf) c[i] = fadd(a.sigmoid ? s[i] : fmul(s[i], most), b);
                if (c[i] > -kInf) size = max(size, fabsf(c[i]));
            }
            err += kStep * warp_max(size);  // the rounding of score + bias
        }
    }
    int id;
    float x = -kInf;
    if (__any_sync(kAll, bad)) {  // a row that cannot be scored: valid experts, and NaN as their weights
        id = lane;
    } else {
        bool unsure = false;
        id = choose<ELT, VPL, float>(a, t, lane, c, err, unsure);
        if (__any_sync(kAll, unsure)) id = choose64<ELT, VPL>(a, t, lane);
        if (id >= 0) x = logit<ELT>(a, t, id);
    }
    const Chosen chosen(x, a.sigmoid);
    float w;
    if (a.renorm) {
        w = chosen.u > 0.0f ? fmul(a.scale, fdiv(chosen.u, chosen.sum)) : 0.0f;
    } else if (a.sigmoid) {
        w = x == -kInf ? 0.0f : fmul(a.scale, Sigmoid(x).s);
    } else {
        w = x == -kInf ? 0.0f : fmul(a.scale, fdiv(exp_neg(m - x), total));
    }
    if (__any_sync(kAll, bad)) w = __uint_as_float(0x7FC00000u);
    if (lane < a.topk) {
        a.ids[t * a.topk + lane] = id;
        a.weights[t * a.topk + lane] = w;
    }
}

// d_logits for the gradient g of the weights.  With u_j = s_j / (sum of the
// chosen s): renormalised, d_j = scale u_j (g_j - sum_i g_i u_i), for sigmoid
// times 1 - s_j, and zero for what was not chosen (the softmax's sum cancels);
// else d_e = scale (s_e g_e [chosen] - s_e sum_j g_j s_j) for softmax and scale
// g_j s_j (1 - s_j) for sigmoid.  A warp to a token.
template <Elt ELT, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const __grid_constant__ RouteArgs a) {
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
        float m = -kInf, total = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = max(m, d[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            d[i] = d[i] == -kInf ? 0.0f : exp_neg(m - d[i]);
            total = fadd(total, d[i]);
        }
        const float inv = fdiv(1.0f, lane_sum(total));
        v = x == -kInf ? 0.0f : fmul(g, fmul(exp_neg(m - x), inv));
        const float all = fmul(inv, lane_sum(v));
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = d[i] == 0.0f ? 0.0f : -fmul(d[i], all);
    }
    for (int j = 0; j < a.topk; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        const float add = __shfl_sync(kAll, v, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e == lane * VPL + i) d[i] = fadd(d[i], add);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane * VPL + i < a.E) store_f32<ELT>(a.d_logits, t * a.E + lane * VPL + i, d[i]);
}

template <Elt ELT, int VPL>
cudaError_t launch(bool grad, const RouteArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)ceil_div(a.T, kWarps));
    return grad ? launch_overlapped(route_grad_kernel<ELT, VPL>, grid, kWarps * 32, 0, 0, s, a)
                : launch_overlapped(route_kernel<ELT, VPL>, grid, kWarps * 32, 0, 0, s, a);
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
