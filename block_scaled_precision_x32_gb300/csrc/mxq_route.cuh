// mxq_route.cuh -- a router's logits to experts and weights, and the gradient.
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
// with 48 bits (a few of a thousand tokens), and what those cannot tell with 64.
//
// A warp to a token, VPL consecutive experts to a lane, in registers.  Bound by
// instructions and, for few tokens, by the latency of their chain: 48 x 32 with
// topk 2 take 1.7 us, 65536 x 160 with eight groups 54 us.  From kQuadTokens on
// four lanes take a token where its sizes allow.
#pragma once

#include <type_traits>

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
// A number as the sum of two floats, the second at most half a unit in the
// last place of the first: 48 bits.  (The sums and products are Dekker's and
// Knuth's.)  fp64 units are few here, and each of their results takes a hundred
// clocks.
struct Wide {
    float h, l;
};
__device__ __forceinline__ Wide wide(float h, float l = 0.0f) { return {h, l}; }
__device__ __forceinline__ Wide sum_of(float a, float b) {  // exact
    const float s = fadd(a, b), v = fadd(s, -a);
    return {s, fadd(fadd(a, -fadd(s, -v)), fadd(b, -v))};
}
__device__ __forceinline__ Wide sum_of_ordered(float a, float b) {  // exact for |a| >= |b|
    const float s = fadd(a, b);
    return {s, fadd(b, -fadd(s, -a))};
}
__device__ __forceinline__ Wide add(Wide a, Wide b) {
    const Wide s = sum_of(a.h, b.h);
    return sum_of_ordered(s.h, fadd(s.l, fadd(a.l, b.l)));
}
__device__ __forceinline__ Wide mul(Wide a, Wide b) {
    const float p = fmul(a.h, b.h);
    return sum_of_ordered(p, ffma(a.l, b.h, ffma(a.h, b.l, ffma(a.h, b.h, -p))));
}
__device__ __forceinline__ Wide reciprocal(Wide a) {
    const float y = fdiv(1.0f, a.h);
    return sum_of_ordered(y, fmul(y, ffma(-y, a.l, ffma(-y, a.h, 1.0f))));
}

// exp(-a) for a >= 0, off by 2^-45 of itself.  -a = r - n ln 2 with ln 2 in
// three parts, the first two of which times n are exact; then expm1(r / 16) by
// its series, and (1 + E)^2 - 1 = 2 E + E^2 four times.  A function of its own, and
// loops around it that are not unrolled: what is seldom needed is not in the
// instruction cache, and to fetch it takes longer than to run it.
__device__ __noinline__ Wide exp_neg_wide(Wide a) {
    const bool gone = a.h >= 120.0f;
    if (gone) a = wide(120.0f);
    constexpr float L1 = 45426.0f / 65536.0f, L2 = 0x1.7f7e000000000p-20f, L3 = -0x1.c610ca0000000p-37f;
    const float n = rintf(fmul(a.h, 1.4426950f));
    const Wide s = sum_of(fmul(n, L1), -a.h), t = sum_of(s.h, fmul(n, L2));
    Wide q = sum_of_ordered(t.h, fadd(fadd(s.l, t.l), ffma(n, L3, -a.l)));
    q = {fmul(q.h, 0.0625f), fmul(q.l, 0.0625f)};
    const Wide q2 = mul(q, q), q3 = mul(q2, q);
    const float rest = fmul(fmul(q2.h, q2.h), ffma(q.h, ffma(q.h, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f));
    Wide e = add(add(q, {fmul(q2.h, 0.5f), fmul(q2.l, 0.5f)}), mul(q3, {1.0f / 6.0f, -0x1.5555560000000p-28f}));
    e = sum_of_ordered(e.h, fadd(e.l, rest));
#pragma unroll
    for (int i = 0; i < 4; ++i) e = add({fmul(e.h, 2.0f), fmul(e.l, 2.0f)}, mul(e, e));
    const float half = __uint_as_float((uint32_t)(127 - (int)n / 2) << 23), other = __uint_as_float((uint32_t)(127 - ((int)n - (int)n / 2)) << 23);
    const Wide one = sum_of(1.0f, e.h);
    e = sum_of_ordered(one.h, fadd(one.l, e.l));
    return {gone ? 0.0f : fmul(fmul(e.h, half), other), gone ? 0.0f : fmul(fmul(e.l, half), other)};
}

__device__ __forceinline__ uint64_t key_of(Wide v) { return (uint64_t)key_of(v.h) << 32 | key_of(v.l); }
__device__ __forceinline__ void from_key(uint32_t k, float& v) { v = of_key(k); }
__device__ __forceinline__ void from_key(uint64_t k, Wide& v) { v = {of_key((uint32_t)(k >> 32)), of_key((uint32_t)k)}; }
__device__ __forceinline__ void from_key(uint64_t k, double& v) { v = of_key(k); }

// What the choice needs of a number, fp32, Wide or fp64.
template <typename Real>
__device__ __forceinline__ Real of(float v) {
    return (Real)v;
}
template <>
__device__ __forceinline__ Wide of<Wide>(float v) {
    return wide(v);
}
template <typename Real>
__device__ __forceinline__ bool more(Real a, Real b) { return a > b; }
__device__ __forceinline__ bool more(Wide a, Wide b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
template <typename Real>
__device__ __forceinline__ Real larger(Real a, Real b) { return max(a, b); }
__device__ __forceinline__ Wide larger(Wide a, Wide b) { return more(a, b) ? a : b; }
template <typename Real>
__device__ __forceinline__ Real smaller(Real a, Real b) { return min(a, b); }
__device__ __forceinline__ Wide smaller(Wide a, Wide b) { return more(a, b) ? b : a; }
// (a + b) / 2 for a >= b > -inf, whose halves come first: two of the type's
// largest or lowest numbers do not overflow.  An infinite a is the result itself,
// which the steps of a Wide sum would make a NaN.
__device__ __forceinline__ float half(float a) { return fmul(a, 0.5f); }
__device__ __forceinline__ double half(double a) { return a * 0.5; }
__device__ __forceinline__ Wide half(Wide a) { return {fmul(a.h, 0.5f), fmul(a.l, 0.5f)}; }
__device__ __forceinline__ float half_sum(float a, float b) { return ffma(a, 0.5f, half(b)); }
__device__ __forceinline__ double half_sum(double a, double b) { return half(a) + half(b); }
__device__ __forceinline__ Wide half_sum(Wide a, Wide b) { return a.h == kInf ? a : add(half(a), half(b)); }
template <typename Real>
__device__ __forceinline__ Real lane_xor(Real v, int d) { return __shfl_xor_sync(kAll, v, d); }
__device__ __forceinline__ Wide lane_xor(Wide v, int d) { return {__shfl_xor_sync(kAll, v.h, d), __shfl_xor_sync(kAll, v.l, d)}; }
template <typename Real>
__device__ __forceinline__ Real lane_at(Real v, int src) { return __shfl_sync(kAll, v, src); }
__device__ __forceinline__ Wide lane_at(Wide v, int src) { return {__shfl_sync(kAll, v.h, src), __shfl_sync(kAll, v.l, src)}; }
__device__ __forceinline__ bool none(float v) { return v == -kInf; }
__device__ __forceinline__ bool none(double v) { return v == -(double)kInf; }
__device__ __forceinline__ bool none(Wide v) { return v.h == -kInf; }
__device__ __forceinline__ float gap(float a, float b) { return a - b; }
__device__ __forceinline__ float gap(double a, double b) { return (float)(a - b); }
__device__ __forceinline__ float gap(Wide a, Wide b) { return fadd(fadd(a.h, -b.h), fadd(a.l, -b.l)); }
__device__ __forceinline__ float size_of(float v) { return fabsf(v); }
__device__ __forceinline__ float size_of(double v) { return fabsf((float)v); }
__device__ __forceinline__ float size_of(Wide v) { return fabsf(v.h); }
// The relative error of a sum's last rounding, twice over.
template <typename Real>
constexpr float kRound = 0.0f;
template <>
constexpr float kRound<float> = 1.0f / (1 << 23);
template <>
constexpr float kRound<Wide> = 1.0f / (1ull << 45);

// The two largest of some numbers.
template <typename Real>
struct Top2 {
    Real a = of<Real>(-kInf), b = of<Real>(-kInf);
    __device__ __forceinline__ void add(const Real& v) {
        b = larger(b, smaller(a, v));
        a = larger(a, v);
    }
    __device__ __forceinline__ void add(const Top2& o) {
        b = larger(larger(b, o.b), smaller(a, o.a));
        a = larger(a, o.a);
    }
    __device__ __forceinline__ void merge(int d) {
        Top2 o;
        o.a = lane_xor(a, d);
        o.b = lane_xor(b, d);
        add(o);
    }
    // The group's score, half of it where it is a sum; -inf where no expert of it can be chosen.
    __device__ __forceinline__ Real score(int top) const { return top == 1 ? a : none(b) ? half(a) : half_sum(a, b); }
    // Magnitudes that are rounded in it; what is infinite is exact.
    __device__ __forceinline__ float size() const { return finite_size(size_of(a)) + finite_size(size_of(b)); }
    __device__ __forceinline__ static float finite_size(float v) { return v < kInf ? half(v) : 0.0f; }
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

// Is the lane's group, of 1 << shift lanes, among the best?  mine: its score,
// size: the magnitudes in it; a choice within the error of the scores sets `unsure`.
// The choice is certain if no group's own error takes it across the middle
// between the last group that is kept and the best that is not: a group that a
// bias of -1e9 keeps out has a large error, and is far from it.
template <typename Real>
__device__ __forceinline__ bool kept_group(const RouteArgs& a, int lane, const Real& mine, float size, int group, int shift, float err, bool& unsure) {
    int ahead = 0;
    // a group's lanes share the comparisons with the others
#pragma unroll 1
    for (int g0 = 0; g0 < a.groups; g0 += 1 << shift) {
        const int g = g0 + (lane & ((1 << shift) - 1));
        const Real other = lane_at(mine, (g << shift) & 31);
        const bool less = more(mine, other);
        ahead += g < a.groups && !less && (g < group || more(other, mine)) ? 1 : 0;
    }
    for (int d = 1; d < 1 << shift; d *= 2) ahead += __shfl_xor_sync(kAll, ahead, d);
    const bool real = group < a.groups;
    if (err >= 0.0f && a.topk_groups < a.groups) {
        const unsigned last = __ballot_sync(kAll, real && ahead == a.topk_groups - 1), next = __ballot_sync(kAll, real && ahead == a.topk_groups);
        const Real least = lane_at(mine, __ffs(last) - 1), best = lane_at(mine, __ffs(next) - 1);
        const float from_middle = half(gap(least, best)) + (ahead < a.topk_groups ? gap(mine, least) : gap(best, mine));
        unsure |= real && size_of(least) < kInf && !none(best) && !(from_middle > err + 1.5f * kRound<Real> * size);  // infinite ones are ties, or far ahead
    }
    return real && ahead < a.topk_groups;
}

// Takes the experts of all but the best groups out (c = -inf).
template <int VPL, Groups GROUPS, typename Real>
__device__ __forceinline__ void best_groups(const RouteArgs& a, int lane, Real (&c)[VPL], float err, bool& unsure, float* stage = nullptr) {
    Top2<Real> top;
    int group = lane, shift = 0;
    if constexpr (GROUPS == ANY && std::is_same<Real, float>::value) {
        // through shared memory, as many lanes to a group as there are for each
        shift = a.group_shift;
        group = lane >> shift;
#pragma unroll
        for (int i = 0; i < VPL; ++i) stage[lane * VPL + i] = c[i];
        __syncwarp();
        if (group < a.groups)
            for (int e = group * a.group_size + (lane & ((1 << shift) - 1)); e < (group + 1) * a.group_size; e += 1 << shift) top.add(stage[e]);
        __syncwarp();
#pragma unroll 1
        for (int d = 1; d < 1 << shift; d *= 2) top.merge(d);
    } else if constexpr (GROUPS == LANES) {
        shift = a.group_shift;
        group = lane >> shift;
        top = top2_of<VPL>(c);
#pragma unroll 1
        for (int d = 1; d < 1 << shift; d *= 2) top.merge(d);
    } else {
#pragma unroll 1
        for (int g = 0; g < a.groups; ++g) {
            Top2<Real> of;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (lane * VPL + i >= g * a.group_size && lane * VPL + i < (g + 1) * a.group_size) of.add(c[i]);
#pragma unroll 1
            for (int d = 1; d < 32; d *= 2) of.merge(d);
            if (lane == g) top = of;
        }
    }
    const bool kept = kept_group<Real>(a, lane, top.score(a.group_top), top.size(), group, shift, err, unsure);
    if constexpr (GROUPS == LANES) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = kept ? c[i] : of<Real>(-kInf);
    } else {
        const unsigned mask = __ballot_sync(kAll, kept);
        int g = lane * VPL / a.group_size;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane * VPL + i;
            g += e >= (g + 1) * a.group_size ? 1 : 0;  // the next expert's group is the same or the next
            if (e >= a.E || !(mask >> (g << shift) & 1)) c[i] = of<Real>(-kInf);
        }
    }
}

// Equal logits with equal biases are ties, which the index decides.
template <Elt ELT>
__device__ __forceinline__ bool are_ties(const RouteArgs& a, int64_t t, int e, int f) {
    return key_of(logit<ELT>(a, t, e)) == key_of(logit<ELT>(a, t, f)) && (!a.bias || key_of(a.bias[e]) == key_of(a.bias[f]));
}

// Is c, behind last_c in the order, within the error of the two?  Infinite ones are
// ties, or far ahead of what is finite.
template <typename Real>
__device__ __forceinline__ bool is_near(float err, Real last_c, Real c) {
    return size_of(last_c) < kInf && gap(last_c, c) <= 2 * err + kRound<Real> * max(size_of(last_c), size_of(c));
}

// Can two of the order, last in front of e, not be told apart?  To be asked of
// neighbours among the chosen, and of the last chosen with each that is not: next to
// it may be its ties alone, and behind them what belongs in its place.
template <Elt ELT, typename Real>
__device__ __forceinline__ bool too_near(const RouteArgs& a, int64_t t, float err, Real last_c, int last, Real c, int e) {
    return is_near(err, last_c, c) && !are_ties<ELT>(a, t, last, e);
}

// The topk largest of c, one after the other: lane j's result is the j-th, -1
// for none.  c is -inf for what cannot be chosen.  err: how far a c may be
// off what exact arithmetic gives, besides its last rounding; neighbours that
// cannot be told apart set `unsure`.  A negative err: c is taken as it is.
template <Elt ELT, int VPL, typename Real>
__device__ __forceinline__ int choose_in_turn(const RouteArgs& a, int64_t t, int lane, const Real (&c)[VPL], float err, bool& unsure) {
    using Key = decltype(key_of(Real()));
    Key key[VPL], top = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = none(c[i]) ? (Key)0 : key_of(c[i]);
        top = max(top, key[i]);
    }
    int id = -1, last = -1;
    Real last_c = of<Real>(0.0f);
#pragma unroll 1
    for (int j = 0; j < a.topk; ++j) {
        const Key best = warp_max(top);
        if (best == 0) return id;
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
        if (lane == j) id = e;
        if (err >= 0.0f) {
            Real now;
            from_key(best, now);
            if (j && too_near<ELT>(a, t, err, last_c, last, now, e)) unsure = true;
            last = e;
            last_c = now;
        }
    }
    if (err >= 0.0f) {
        unsigned near = 0;  // of the lane's others, to the last chosen
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            Real other;
            from_key(key[i], other);
            near |= key[i] != 0 && is_near(err, last_c, other) ? 1u << i : 0u;
        }
#pragma unroll 1
        for (; near; near &= near - 1) unsure |= !are_ties<ELT>(a, t, last, lane * VPL + __ffs(near) - 1);
    }
    return id;
}

// A second look, with 48 bits, at the candidates of a token that 24 bits cannot
// put in order: n <= 32 keys in `list`, their lower words the complements of the
// experts' indices, one to a lane.  They come back in their order; false where 48
// bits do not tell either.
template <Elt ELT>
__device__ __noinline__ bool resolve(const RouteArgs& a, int64_t t, int n, uint64_t* list) {
    const int lane = threadIdx.x & 31, id = lane < n ? (int)~(uint32_t)list[lane] : 0;
    const float x = logit<ELT>(a, t, id), b = a.bias ? a.bias[id] : 0.0f;
    float m = 0.0f, most = 1.0f;
    Wide sum = wide(0.0f), c;
    if (!a.sigmoid) {
        m = -kInf;
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) m = max(m, logit<ELT>(a, t, e));
        __syncwarp();
        m = warp_max(m);
    }
    // the softmax's sum takes each lane through its experts; the last step is the candidate's own
#pragma unroll 1
    for (int e = a.sigmoid ? a.E : 0;; e += 32) {
        const bool last = e >= a.E, there = e + lane < a.E;
        const float v = last ? x : there ? logit<ELT>(a, t, e + lane) : -kInf;
        c = exp_neg_wide(a.sigmoid ? wide(fabsf(v)) : v == -kInf ? wide(kExpEnd) : sum_of(m, -v));
        if (last) break;
        sum = add(sum, c);
    }
    if (a.sigmoid) {
        const Wide inv = reciprocal(add(wide(1.0f), c));
        c = x < 0.0f ? mul(c, inv) : inv;
    } else {
#pragma unroll 1
        for (int d = 16; d; d /= 2) sum = add(sum, lane_xor(sum, d));
        sum = reciprocal(sum);
        most = sum.h;
        c = mul(c, sum);
    }
    if (a.bias) c = fabsf(b) < kInf ? add(c, wide(b)) : wide(b);
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const Wide o = lane_at(c, j);
        const int other = __shfl_sync(kAll, id, j);
        rank += more(o, c) || (!more(c, o) && other < id) ? 1 : 0;
    }
    // each place's number, then each place's expert: those of neighbours are compared as too_near has to be asked
    const float err = most * (1.0f / (1ull << 41));  // 2^-45 of the exponential, the sum, the quotient and the product
    __syncwarp();
    if (lane < n) list[rank] = (uint64_t)__float_as_uint(c.h) << 32 | __float_as_uint(c.l);
    __syncwarp();
    const auto at = [&](int place) { return wide(__uint_as_float((uint32_t)(list[place] >> 32)), __uint_as_float((uint32_t)list[place])); };
    const int front = min(lane, a.topk) - 1;
    bool unsure = lane && lane < n && is_near(err, at(front), at(lane));
    __syncwarp();
    if (lane < n) list[rank] = (uint64_t)key_of(c.h) << 32 | (uint32_t)~id;
    __syncwarp();
    if (unsure) unsure = !are_ties<ELT>(a, t, (int)~(uint32_t)list[front], (int)~(uint32_t)list[lane]);
    return !__any_sync(kAll, unsure);
}

// The same for fp32 in fewer steps.  The topk + 1 largest are among the values
// that reach the (topk + 1)-th largest of the lanes' own largest ones: a dozen
// for topk 8.  Those go to shared memory, one to a lane, and each counts how
// many are ahead of it.  More than 32 of them are chosen in turn.  Candidates
// that cannot be told apart get their second look here.
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
    if (err >= 0.0f) from -= 2 * err + kRound<float> * fabsf(from);  // what may be ahead of it
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
    if (err >= 0.0f) {
        bool near = false;
        if (lane && lane < n) {
            const uint64_t k = list[min(lane, a.topk) - 1], l = list[lane];
            near = too_near<ELT>(a, t, err, of_key((uint32_t)(k >> 32)), (int)~(uint32_t)k, of_key((uint32_t)(l >> 32)), (int)~(uint32_t)l);
        }
        if (__any_sync(kAll, near)) unsure |= !resolve<ELT>(a, t, n, list);
    }
    return lane < a.topk && lane < n ? (int)~(uint32_t)list[lane] : -1;
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

// Are the lane's logits all `v`?
template <int VPL>
__device__ __forceinline__ bool alike(const RouteArgs& a, int lane, const float (&x)[VPL], float v) {
    bool same = true;
#pragma unroll
    for (int i = 0; i < VPL; ++i) same &= x[i] == v || lane * VPL + i >= a.E;
    return same;
}

// Scores of N logits: 1 / (1 + exp(-x)), or exp(x - m) for the softmax.  The
// product with log2(e) is rounded once, which makes the exponential off by |x| units
// of 2^-24 of itself: times s (1 - s), or its own value, that is less than one, which
// is all that a comparison of scores needs, and the sum of a softmax.  The dense
// gradient takes its probabilities from here as well: the small ones are off by up to
// twice |x - m| units of themselves (x - m is rounded too): 28 on 65536 x 256 logits of
// N(0, 1) and their like, where exp_neg leaves 17, and 6.1e-8 against 5.0e-8 in the norm.
// That is less than a rounding of the largest one, and saves 1 us of 24.  -inf gives 0.
constexpr float kLog2e = 1.4426950216293335f;
template <int N>
__device__ __forceinline__ void scores(const RouteArgs& a, const float (&x)[N], float m, float (&s)[N]) {
    const float from = m == -kInf ? 0.0f : m;  // a row of -inf alone
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const int j = N > 1 ? i + 1 : i;
        if (a.sigmoid) {
            const float2 t = mul2(make_float2(x[i], x[j]), both(-kLog2e));
            const float2 d = fma2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), both(1.0f), both(1.0f));
            s[i] = rcp_approx(d.x);
            s[j] = rcp_approx(d.y);
        } else {
            const float2 t = mul2(make_float2(x[i] - from, x[j] - from), both(kLog2e));
            s[i] = ex2_approx(t.x);
            s[j] = ex2_approx(t.y);
        }
    }
}

// A second look with 48 bits at a whole token, whose best groups 24 cannot tell;
// -2 where those do not tell either.
template <Elt ELT, int VPL, Groups GROUPS>
__device__ __noinline__ int choose48(const RouteArgs& a, int64_t t, int lane) {
    float x[VPL];
    load_logits<ELT, VPL>(a, t, lane, x);
    float m = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = max(m, x[i]);
    m = warp_max(m);
    Wide c[VPL], sum = wide(0.0f);
#pragma unroll 1
    for (int i = 0; i < VPL; ++i) {
        const Wide e = exp_neg_wide(a.sigmoid ? wide(fabsf(x[i])) : sum_of(m, -x[i]));
        if (a.sigmoid) {
            const Wide inv = reciprocal(add(wide(1.0f), e));
            c[i] = x[i] < 0.0f ? mul(e, inv) : inv;
        } else {
            c[i] = x[i] == -kInf ? wide(0.0f) : e;
            sum = add(sum, c[i]);
        }
    }
    float most = 1.0f;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int d = 16; d; d /= 2) sum = add(sum, lane_xor(sum, d));
        sum = reciprocal(sum);
        most = sum.h;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (!a.sigmoid) c[i] = mul(c[i], sum);
        const int e = lane * VPL + i;
        if (a.bias && e < a.E) {
            const float b = a.bias[e];
            c[i] = fabsf(b) < kInf ? add(c[i], wide(b)) : wide(b);
        }
        if (x[i] == -kInf) c[i] = wide(-kInf);
    }
    bool unsure = false;
    const float err = most * (1.0f / (1ull << 41));  // as above
    if constexpr (GROUPS != NONE) best_groups<VPL, GROUPS, Wide>(a, lane, c, err, unsure);
    const int id = choose_in_turn<ELT, VPL, Wide>(a, t, lane, c, err, unsure);
    return __any_sync(kAll, unsure) ? -2 : id;
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
    // four at a time: each takes thousands of clocks, most of them waiting
    double c[VPL], sum = 0.0;
#pragma unroll 4
    for (int i = 0; i < VPL; ++i) {
        c[i] = exp(a.sigmoid ? -(double)x[i] : (double)x[i] - (double)m);
        if (a.sigmoid) c[i] = 1.0 / (1.0 + c[i]);
        sum += c[i];
    }
    if (!a.sigmoid) {
        for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(kAll, sum, d);
        sum = 1.0 / sum;
    }
#pragma unroll 4
    for (int i = 0; i < VPL; ++i) {
        if (!a.sigmoid) c[i] *= sum;
        if (a.bias && lane * VPL + i < a.E) c[i] += (double)a.bias[lane * VPL + i];
        if (x[i] == -kInf) c[i] = -(double)kInf;
    }
    bool unsure = false;
    if constexpr (GROUPS != NONE) best_groups<VPL, GROUPS, double>(a, lane, c, -1.0f, unsure);
    return choose_in_turn<ELT, VPL, double>(a, t, lane, c, -1.0f, unsure);
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

// One token to a warp, from its logits to its outputs.
template <Elt ELT, int VPL, Groups GROUPS>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int lane, uint64_t* list, float* stage = nullptr) {
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
            // in units of 2^-24 of the largest score.  Sigmoid: 1 of the exponential, 1 of the sum, 2 of the reciprocal.  Softmax: 3
            // of the exponential; of the sum 3, its VPL + 4 additions and 2.3 ln E of what the exponentials are off by; 2 of the rest
            const float most = a.sigmoid ? 1.0f : fdiv(1.0f, total);
            err = (a.sigmoid ? 6.0f : VPL + 32.0f) * 5.9604645e-8f * most;
            // all experts alike, as those of a padded row or of a router that has learned nothing: ties, which need no second look
            bool same = __all_sync(kAll, alike<VPL>(a, lane, c, __shfl_sync(kAll, c[0], 0)));
            float b[VPL];
#pragma unroll
            for (int i = 0; i < VPL; ++i) b[i] = 0.0f;
            if (a.bias) {
                load_bias<VPL>(a, lane, b);
                const float top = max_nan<VPL>(b);
                bad |= top != top;
                if (same) same = __all_sync(kAll, alike<VPL>(a, lane, b, __shfl_sync(kAll, b[0], 0)));
            }
            if (same) err = -1.0f;
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
        if constexpr (GROUPS != NONE) best_groups<VPL, GROUPS, float>(a, lane, c, err, unsure, stage);
        id = choose32<ELT, VPL>(a, t, lane, c, err, unsure, list);
        if (__any_sync(kAll, unsure)) {
            id = choose48<ELT, VPL, GROUPS>(a, t, lane);
            if (id == -2) id = choose64<ELT, VPL, GROUPS>(a, t, lane);
        }
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

template <Elt ELT, int VPL, Groups GROUPS>
__global__ void __launch_bounds__(kWarps * 32, VPL == 8 ? 9 : 0) route_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ __align__(16) uint64_t lists[kWarps][32];
    __shared__ float stages[GROUPS == ANY ? kWarps : 1][GROUPS == ANY ? 32 * VPL : 1];
    let_next_start();
    wait_for_stream();
    const int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (t < a.T) route_token<ELT, VPL, GROUPS>(a, t, threadIdx.x & 31, lists[threadIdx.x / 32], stages[GROUPS == ANY ? threadIdx.x / 32 : 0]);
}

// ---- many tokens: four lanes to one
//
// Of a warp's work for a token the larger part is done for a dozen candidates
// or for nine rounds, in which most lanes only wait.  Here eight tokens share
// a warp: lane l of a token's four has the chunks l, l + 4, ... of four experts
// each, J of them, in registers.  The steps are the same:
//   - a group is JG chunks of each lane; every lane knows all groups' scores;
//   - the ninth largest of the chunks' maxima bounds the candidates: each lane
//     sorts its own, and two exchanges merge the four lists;
//   - each lane appends its candidates to a list, the lists are put together,
//     and a candidate's rank is the number of those ahead of it.
// Groups and candidates that 24 bits cannot put in order are looked at again by
// the whole warp, and the token goes on.  One with anything else unusual (NaN,
// groups that 48 bits cannot tell apart either, kSlots candidates in a lane or more
// than kRanked) is left to the whole warp, which then takes it by itself, unless all
// experts are alike, as in a padded row (65536 tokens, half of them zeros, take 100
// us, 150 one by one).  Each of
// these holds the warp up for 5 to 10 us: without any of them the largest case
// below would take 41 us.  kSlots 8, which three of a thousand random tokens meet,
// took it from 50 to 52.  For topk up to 8.
//
// 65536 x 256 fp32 with sigmoid, a bias and groups take 48 us, where their 71 MB
// would take 11 (a warp to each took 68); bf16 softmax without groups 22.  Bound
// by instructions, about 440 a token, which the instruction cache delivers at
// half the rate they could start at: all of it is unrolled, so that the scores
// stay in registers.  96 registers, 20 warps a multiprocessor in blocks of one
// (16: 49 us; 18, 21 and more, whose registers spill: 54 to 63; blocks of two or
// four warps: 50).
constexpr int kQuadTopk = 8, kQuadKept = kQuadTopk + 1, kSlots = 12, kRanked = 28;
constexpr int64_t kQuadTokens = 16384;  // from here on it is the faster one, but for what launch leaves out
constexpr int kQuadWarps = 1;  // a warp that looks twice at a token keeps no others from making room

__device__ __forceinline__ void order(float& a, float& b) {  // the larger one first
    const float t = max(a, b);
    b = min(a, b);
    a = t;
}

template <Elt ELT>
__device__ __forceinline__ float4 load_chunk(const RouteArgs& a, int64_t t, int chunk) {
    if constexpr (ELT == Elt::FP32) {
        return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + t * a.ld) + chunk);
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + t * a.ld) + chunk);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    }
}

// What 24 bits tell of the groups of a token with each one's own error: a bit for
// each that is kept, -1 where they do not tell.  The four lanes have registers for
// the largest error alone (with each group's in them the usual call took 50 us
// instead of 48), which a group that a bias of -1e9 keeps out sets for every token:
// 65536 x 256 take 99 us then, and 315 if all of them go on to 48 bits.
template <Elt ELT, int VPL>
__device__ __noinline__ int groups24(const RouteArgs& a, int64_t t, int lane) {
    float c[VPL], s[VPL], b[VPL], total = 0.0f, most = 1.0f;
    load_logits<ELT, VPL>(a, t, lane, c);
    scores<VPL>(a, c, a.sigmoid ? 0.0f : warp_max(max_nan<VPL>(c)), s);
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) total = fadd(total, s[i]);
        most = fdiv(1.0f, lane_sum(total));
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) b[i] = 0.0f;
    if (a.bias) load_bias<VPL>(a, lane, b);
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = c[i] > -kInf ? ffma(s[i], most, b[i]) : -kInf;
    Top2<float> top = top2_of<VPL>(c);
    const int shift = a.group_shift;
#pragma unroll 1
    for (int d = 1; d < 1 << shift; d *= 2) top.merge(d);
    bool unsure = false;
    const float err = (a.sigmoid ? 6.0f : VPL + 32.0f) * 5.9604645e-8f * most;  // as in route_token
    const unsigned lanes = __ballot_sync(kAll, kept_group<float>(a, lane, top.score(a.group_top), top.size(), lane >> shift, shift, err, unsure));
    int bits = 0;
    for (int g = 0; g < a.groups; ++g) bits |= (int)(lanes >> (g << shift) & 1) << g;
    return __any_sync(kAll, unsure) ? -1 : bits;
}

// A second look, with 48 bits, at the groups of a token: a bit for each that is
// kept, -1 where 48 bits do not tell either.  Only what can be among the largest of
// its group gets one.
template <Elt ELT, int VPL>
__device__ __noinline__ int groups48(const RouteArgs& a, int64_t t, int lane) {
    float c[VPL], b[VPL];
    load_logits<ELT, VPL>(a, t, lane, c);
    float m = max_nan<VPL>(c), most = 1.0f;
    Wide sum = wide(0.0f);
    const bool same = __all_sync(kAll, alike<VPL>(a, lane, c, __shfl_sync(kAll, c[0], 0)));
    if (same) return -1;  // most likely ties
    if (!a.sigmoid) {
        m = warp_max(m);
#pragma unroll 1
        for (int e = lane; e < a.E; e += 32) {
            const float x = logit<ELT>(a, t, e);
            sum = add(sum, exp_neg_wide(x == -kInf ? wide(kExpEnd) : sum_of(m, -x)));
        }
        __syncwarp();
#pragma unroll 1
        for (int d = 16; d; d /= 2) sum = add(sum, lane_xor(sum, d));
        sum = reciprocal(sum);
        most = sum.h;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) b[i] = 0.0f;
    if (a.bias) load_bias<VPL>(a, lane, b);
    {
        float s[VPL];
        scores<VPL>(a, c, m, s);
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = c[i] > -kInf ? ffma(s[i], most, b[i]) : -kInf;
    }
    Top2<float> top = top2_of<VPL>(c);
    const int shift = a.group_shift, group = lane >> shift;
#pragma unroll 1
    for (int d = 1; d < 1 << shift; d *= 2) top.merge(d);
    const float last = a.group_top == 1 ? top.a : top.b, err = (a.sigmoid ? 6.0f : VPL + 32.0f) * 5.9604645e-8f * most,
                from = last - (2 * err + kRound<float> * fabsf(last));
    unsigned may = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) may |= c[i] >= from && c[i] > -kInf ? 1u << i : 0u;
    Top2<Wide> best;
#pragma unroll 1
    while (__any_sync(kAll, may != 0)) {
        const int e = may ? lane * VPL + __ffs(may) - 1 : 0;
        const float x = logit<ELT>(a, t, e), bias = a.bias ? a.bias[e] : 0.0f;
        Wide v = exp_neg_wide(a.sigmoid ? wide(fabsf(x)) : x == -kInf ? wide(kExpEnd) : sum_of(m, -x));
        if (a.sigmoid) {
            const Wide inv = reciprocal(add(wide(1.0f), v));
            v = x < 0.0f ? mul(v, inv) : inv;
        } else {
            v = mul(v, sum);
        }
        if (a.bias) v = add(v, wide(bias));
        if (may) best.add(v);
        may &= may - 1;
    }
#pragma unroll 1
    for (int d = 1; d < 1 << shift; d *= 2) best.merge(d);
    bool unsure = false;
    const bool kept = kept_group<Wide>(a, lane, best.score(a.group_top), best.size(), group, shift, most * (1.0f / (1ull << 41)), unsure);  // as in resolve
    const unsigned lanes = __ballot_sync(kAll, kept);
    int bits = 0;
    for (int g = 0; g < a.groups; ++g) bits |= (int)(lanes >> (g << shift) & 1) << g;
    return __any_sync(kAll, unsure) ? -1 : bits;
}

// Are all logits of the token of these four lanes one number, and all biases one?
template <Elt ELT>
__device__ __noinline__ bool alike_row(const RouteArgs& a, int64_t t) {
    const int lane = threadIdx.x & 31;
    const float x = logit<ELT>(a, t, 0), b = a.bias ? a.bias[0] : 0.0f;
    // as patterns: subnormal numbers are not zeros
    const auto is = [](float v, float w) { return __float_as_uint(v) == __float_as_uint(w); };
    bool same = fabsf(x) < kInf && fabsf(b) < kInf && is(logit<ELT>(a, t, 1 + (lane & 3)), x);
    if (!__any_sync(kAll, same)) return false;  // most often
#pragma unroll 4
    for (int chunk = lane & 3; chunk * 4 < a.E; chunk += 4) {
        const float4 v = load_chunk<ELT>(a, t, chunk);
        same &= is(v.x, x) && is(v.y, x) && is(v.z, x) && is(v.w, x);
        if (a.bias) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(a.bias) + chunk);
            same &= is(c.x, b) && is(c.y, b) && is(c.z, b) && is(c.w, b);
        }
    }
    __syncwarp();
    return (__ballot_sync(kAll, same) >> (lane & 28) & 15) == 15;
}

template <Elt ELT, int J, int JG>
__device__ __noinline__ void route_left(const RouteArgs& a, unsigned left, int64_t t, int lane, uint64_t* list) {
    for (; left; left &= left - 1) {
        __syncwarp();
        route_token<ELT, J / 2, JG ? LANES : NONE>(a, __shfl_sync(kAll, t, __ffs(left) - 1), lane, list);
    }
}

template <Elt ELT, int J, int JG>
__global__ void __launch_bounds__(kQuadWarps * 32, 20 / kQuadWarps) route_quad_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ __align__(16) uint64_t lists[kQuadWarps][8][4 * kSlots];
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31, l = lane & 3;
    const int64_t t0 = ((int64_t)blockIdx.x * kQuadWarps + threadIdx.x / 32) * 8;
    bool strange = false;  // a bias of NaN, or of infinity: tokens are left to the whole warp
    if (a.bias) {
        for (int e = threadIdx.x; e < a.E; e += kQuadWarps * 32) strange |= !(__ldg(a.bias + e) < kInf);
        strange = __syncthreads_or(strange);
    }
    if (t0 >= a.T) return;
    const bool real = t0 + (lane >> 2) < a.T;
    const int64_t t = real ? t0 + (lane >> 2) : a.T - 1;
    uint64_t* list = lists[threadIdx.x / 32][lane >> 2];
    float c[4 * J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const float4 v = (l + 4 * j) * 4 < a.E ? load_chunk<ELT>(a, t, l + 4 * j) : make_float4(-kInf, -kInf, -kInf, -kInf);
        c[4 * j] = v.x, c[4 * j + 1] = v.y, c[4 * j + 2] = v.z, c[4 * j + 3] = v.w;
    }
    float m = max_nan<4 * J>(c);
    bool left = strange || m != m;  // to the whole warp
    if (!a.sigmoid) {
#pragma unroll
        for (int d = 1; d < 4; d *= 2) m = max(m, __shfl_xor_sync(kAll, m, d));
        left |= !(fabsf(m) < kInf);
    }
    const bool scored = a.bias || (JG && a.group_top > 1);
    float total = 0.0f, err = -1.0f;
    if (scored || !(a.sigmoid || a.renorm)) {
        float most = 1.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {  // in place: there are no registers for the logits and the scores
            float(&x)[4] = reinterpret_cast<float(&)[4]>(c[4 * j]);
            float z[4];
            scores<4>(a, x, m, z);
            total = fadd(total, fadd(fadd(z[0], z[1]), fadd(z[2], z[3])));
            if (scored)
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = x[q] > -kInf ? z[q] : -kInf;
        }
        if (!a.sigmoid) {
#pragma unroll
            for (int d = 1; d < 4; d *= 2) total = fadd(total, __shfl_xor_sync(kAll, total, d));
            most = fdiv(1.0f, total);
        }
        if (scored) {
            // as in route_token, with the J + 4 additions of a quad's sum and ln 256
            err = (a.sigmoid ? 6.0f : J + 28.0f) * 5.9604645e-8f * most;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (a.bias && (l + 4 * j) * 4 < a.E) b = __ldg(reinterpret_cast<const float4*>(a.bias) + l + 4 * j);
                c[4 * j] = ffma(c[4 * j], most, b.x), c[4 * j + 1] = ffma(c[4 * j + 1], most, b.y);
                c[4 * j + 2] = ffma(c[4 * j + 2], most, b.z), c[4 * j + 3] = ffma(c[4 * j + 3], most, b.w);
            }
        }
    }
    bool out[JG ? J / JG : 1] = {};  // a group that is not kept
    if constexpr (JG > 0) {
        constexpr int G = J / JG;
        float score[G];
        float size = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            Top2<float> top = top2_of<4 * JG>(c + 4 * JG * g);
            top.merge(1);
            top.merge(2);
            score[g] = top.score(a.group_top);
            size = max(size, top.size());
        }
        float least = kInf, next = -kInf;
        bool kept[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            int ahead = 0;
#pragma unroll
            for (int o = 0; o < G; ++o)
                if (o != g) ahead += (o < g ? score[o] >= score[g] : score[o] > score[g]) ? 1 : 0;
            kept[g] = ahead < a.topk_groups;
            least = kept[g] ? min(least, score[g]) : least;
            next = kept[g] ? next : max(next, score[g]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) out[g] = !kept[g];
        if (scored) {  // the same for every lane, as err is not: a row that cannot be scored has NaN there
            unsigned nears = __ballot_sync(kAll, next > -kInf && least - next <= 2 * err + 3 * kRound<float> * size && !left);
            if (nears) {
                left |= alike_row<ELT>(a, t);
                nears &= __ballot_sync(kAll, !left);
            }
            while (nears) {  // one token after the other, by the whole warp
                const int quad = (__ffs(nears) - 1) >> 2;
                const int64_t token = __shfl_sync(kAll, t, 4 * quad);
                int bits = __shfl_sync(kAll, size, 4 * quad) > 16.0f ? groups24<ELT, J / 2>(a, token, lane) : -1;
                if (bits < 0) bits = groups48<ELT, J / 2>(a, token, lane);
                if (lane >> 2 == quad) {
                    left |= bits < 0;
#pragma unroll
                    for (int g = 0; g < G; ++g) out[g] = !(bits >> g & 1);
                }
                nears &= ~(15u << (4 * quad));
            }
        }
    }
    // the lane's chunks' maxima in descending order, the largest kQuadKept of them
    float from;
    {
        float top[kQuadKept];
#pragma unroll
        for (int i = 0; i < kQuadKept; ++i) top[i] = -kInf;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float v = max(max(c[4 * j], c[4 * j + 1]), max(c[4 * j + 2], c[4 * j + 3]));
            if (JG && out[JG ? j / JG : 0]) v = -kInf;
#pragma unroll
            for (int i = 0; i < kQuadKept && i <= j; ++i) order(top[i], v);
        }
        // the largest of two descending lists are the larger ones of a value and its counterpart from the other list's end
        float both_[kQuadKept], sorted[kQuadKept];
#pragma unroll
        for (int i = 0; i < kQuadKept; ++i) both_[i] = max(top[i], __shfl_xor_sync(kAll, top[kQuadKept - 1 - i], 1));
#pragma unroll
        for (int j = 0; j < kQuadKept; ++j) {
            float v = both_[j];
            sorted[j] = -kInf;
#pragma unroll
            for (int i = 0; i <= j; ++i) order(sorted[i], v);
        }
        from = kInf;
#pragma unroll
        for (int i = 0; i < kQuadKept; ++i) from = min(from, max(sorted[i], __shfl_xor_sync(kAll, sorted[kQuadKept - 1 - i], 2)));
        if (err >= 0.0f) from -= 2 * err + kRound<float> * fabsf(from);  // what may be ahead of it
        from = max(from, -3.4028235e38f);
    }
    int at = 0;
    float2* mine = reinterpret_cast<float2*>(list) + l * kSlots;
#pragma unroll
    for (int i = 0; i < 4 * J; ++i)
        if (c[i] >= (JG && out[JG ? i / (4 * JG) : 0] ? __uint_as_float(0x7FC00000u) : from) && at < kSlots) mine[at++] = make_float2(c[i], __uint_as_float(((l + 4 * (i / 4)) * 4 + i % 4)));
    left |= at == kSlots;
    at = min(at, kSlots - 1);
    // the four lists one behind the other, as keys: by value, then the lower index first
    uint64_t key[kSlots - 1];
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) {
        key[i] = 0;
        if (i < at) {
            const float2 v = mine[i];
            key[i] = (uint64_t)key_of(v.x) << 32 | ~__float_as_uint(v.y);
        }
    }
    int before = at, n = at;
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
        const int other = __shfl_xor_sync(kAll, n, d);
        before += l & d ? other : 0;
        n += other;
    }
    before -= at;
    left |= n > kRanked;
    n = min(n, kRanked);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i)
        if (i < at) list[before + i] = key[i];
    __syncwarp();  // with more than kRanked this lies over one of them
    if (l == 0) list[n] = 0;  // the ranks are counted two at a time
    __syncwarp();
    uint64_t own[kRanked / 4];
    int rank[kRanked / 4];
#pragma unroll
    for (int r = 0; r < kRanked / 4; ++r) {
        own[r] = 0, rank[r] = 0;
        if (__any_sync(kAll, l + 4 * r < n)) {
            own[r] = l + 4 * r < n ? list[l + 4 * r] : 0;
            for (int j = 0; j < n; j += 2) {
                const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(list + j);
                rank[r] += (k.x > own[r] ? 1 : 0) + (k.y > own[r] ? 1 : 0);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRanked / 4; ++r)
        if (l + 4 * r < n) list[rank[r]] = own[r];
    __syncwarp();
    left = __ballot_sync(kAll, left) >> (lane & 28) & 15;  // of one of the four, of all
    if (scored) {
        bool near = false, edge = false;  // edge: the first that is not chosen is near to the last that is
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int place = l + 4 * r;
            if (place < a.topk && place + 1 < n) {
                const uint64_t k = list[place], o = list[place + 1];
                if (is_near(err, of_key((uint32_t)(k >> 32)), of_key((uint32_t)(o >> 32)))) {
                    if (place + 1 == a.topk) edge = true;
                    else near |= !are_ties<ELT>(a, t, (int)~(uint32_t)k, (int)~(uint32_t)o);
                }
            }
        }
        unsigned nears = __ballot_sync(kAll, (near || edge) && !left);
        if (nears) {
            if (__ballot_sync(kAll, edge) >> (lane & 28) & 15)
                for (int place = a.topk + l; place < n; place += 4) {
                    const uint64_t k = list[a.topk - 1], o = list[place];
                    near |= too_near<ELT>(a, t, err, of_key((uint32_t)(k >> 32)), (int)~(uint32_t)k, of_key((uint32_t)(o >> 32)), (int)~(uint32_t)o);
                }
            __syncwarp();
            nears = __ballot_sync(kAll, near && !left);
        }
        while (nears) {  // one token after the other, by the whole warp
            const int quad = (__ffs(nears) - 1) >> 2;
            const bool ok = resolve<ELT>(a, __shfl_sync(kAll, t, 4 * quad), __shfl_sync(kAll, n, 4 * quad), lists[threadIdx.x / 32][quad]);
            left |= !ok && lane >> 2 == quad;
            nears &= ~(15u << (4 * quad));
        }
    }
    int id[2];
    float x[2], w[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int place = l + 4 * r;
        id[r] = place < a.topk && place < n ? (int)~(uint32_t)list[place] : -1;
        x[r] = id[r] >= 0 ? logit<ELT>(a, t, id[r]) : -kInf;
        w[r] = x[r] == -kInf ? 0.0f : a.sigmoid ? Sigmoid(x[r]).s : exp_neg(m - x[r]);
    }
    float sum = fadd(w[0], w[1]);
#pragma unroll
    for (int d = 1; d < 4; d *= 2) sum = fadd(sum, __shfl_xor_sync(kAll, sum, d));
    if (!a.renorm) sum = a.sigmoid ? 1.0f : total;
    else left |= sum < 1e-3f;  // the chosen scores are small, or underflow
    left = __ballot_sync(kAll, left) >> (lane & 28) & 15;
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (real && !left && l + 4 * r < a.topk) {
            a.ids[t * a.topk + l + 4 * r] = id[r];
            a.weights[t * a.topk + l + 4 * r] = fmul(a.scale, fdiv(w[r], sum));
        }
    unsigned again = __ballot_sync(kAll, left && real && l == 0);
    if (again) {
        // all experts alike, as those of a padded row: the first ones are chosen
        const bool same = alike_row<ELT>(a, t);
        const float first = logit<ELT>(a, t, 0),
                    share = a.renorm ? fdiv(1.0f, (float)a.topk) : a.sigmoid ? Sigmoid(first).s : fdiv(1.0f, (float)a.E);
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (left && same && real && l + 4 * r < a.topk) {
                a.ids[t * a.topk + l + 4 * r] = l + 4 * r;
                a.weights[t * a.topk + l + 4 * r] = fmul(a.scale, share);
            }
        again = __ballot_sync(kAll, left && !same && real && l == 0);
    }
    if (again) route_left<ELT, J, JG>(a, again, t, lane, lists[threadIdx.x / 32][0]);
}

// d_logits for the gradient g of the weights.  With u_j = s_j / (sum of the
// chosen s): renormalised, d_j = scale u_j (g_j - sum_i g_i u_i), for sigmoid
// times 1 - s_j, and zero for what was not chosen (the softmax's sum cancels);
// else d_e = scale (s_e g_e [chosen] - s_e sum_j g_j s_j) for softmax and scale
// g_j s_j (1 - s_j) for sigmoid.  A warp to a token; the row is put together in
// shared memory, where a choice finds its expert, and leaves in 16-byte words.
// Bound by HBM: 65536 x 256 fp32 with the whole softmax's gradient 22.8 us for
// 138 MB (6.0 TB/s), with four fifths of the issue slots taken.
template <Elt ELT, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ __align__(16) float rows[kWarps][32 * VPL];
    let_next_start();
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= a.T) return;
    const bool dense = !a.sigmoid && !a.renorm;
    float d[VPL], v;
    if (dense) load_logits<ELT, VPL>(a, t, lane, d);  // ahead of what has to wait for the ids
    int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
    float g = lane < a.topk ? a.g[t * a.topk + lane] : 0.0f;
    if (id < 0 || id >= a.E) id = -1, g = 0.0f;
    g = fmul(a.scale, g);
    const float x = id >= 0 ? logit<ELT>(a, t, id) : -kInf;
    if (!dense) {
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
    a.group_size = a.E / a.groups;
    if constexpr (VPL == 4 || VPL == 8) {
        const bool chunks = a.E % 4 == 0 && on_bytes(a.logits, 16) && (a.T <= 1 || a.ld % 4 == 0) && on_bytes(a.bias, 16);
        // kept experts of so few chunks that no bound is found among the chunks' maxima, and more of them than can be ranked: every token
        // would be left to the whole warp after all.  32 kept in two groups or one, 65536 x 128: 125 and 121 us, a warp to each 47 and 48;
        // 65536 x 256: 193 and 167, a warp to each 76 and 68
        const int kept = a.groups > 1 ? a.topk_groups * a.group_size : a.E;
        const bool crowded = kept > kRanked && kept < 4 * kQuadKept;
        if (chunks && !crowded && a.topk <= kQuadTopk && a.T >= kQuadTokens) {
            constexpr int J = 2 * VPL;
            const dim3 grid((unsigned)ceil_div(a.T, kQuadWarps * 8));
            if (a.groups == 1) return launch_overlapped(route_quad_kernel<ELT, J, 0>, grid, kQuadWarps * 32, 0, 0, s, a);
            for (a.group_shift = 0; VPL << a.group_shift < a.group_size;) ++a.group_shift;
            if (a.group_size == 16) return launch_overlapped(route_quad_kernel<ELT, J, 1>, grid, kQuadWarps * 32, 0, 0, s, a);
            if (a.group_size == 32) return launch_overlapped(route_quad_kernel<ELT, J, 2>, grid, kQuadWarps * 32, 0, 0, s, a);
        }
    }
    if (a.groups == 1) return launch_overlapped(route_kernel<ELT, VPL, NONE>, grid, kWarps * 32, 0, 0, s, a);
    if constexpr (VPL <= 8)  // more experts than 256 go the general way
        for (int shift = 0; shift < 6; ++shift)
            if (VPL << shift == a.group_size) {
                a.group_shift = shift;
                return launch_overlapped(route_kernel<ELT, VPL, LANES>, grid, kWarps * 32, 0, 0, s, a);
            }
    for (a.group_shift = 0; a.groups << (a.group_shift + 1) <= 32;) ++a.group_shift;
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

// The launches of one type of logits: a translation unit for each, which
// compile side by side.
template <Elt ELT>
cudaError_t route_launch(bool grad, const RouteArgs& a, cudaStream_t s) {
    const cudaError_t e = launch<ELT>(grad, a, s);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

}  // namespace
}  // namespace mxq
