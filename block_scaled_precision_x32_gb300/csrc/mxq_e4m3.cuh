// mxq_e4m3.cuh -- what the kernels share that write E4M3 with one power-of-two
// scale per 128 elements, and that work on rows of units of 16 elements.
//
// For a block with largest magnitude amax = (1 + f) 2^E the scale is the
// least power of two that keeps amax / 2^s within E4M3's largest value
// 448 = 1.75 * 2^8: s = E - 8, and one more if f > 0.75.
#pragma once

#include "mxq_device.cuh"
#include "mxq_internal.h"

namespace mxq {

// UE8M0 code of a block from the bits of its fp32 amax; 255 for NaN and Inf.
__device__ __forceinline__ uint32_t scale_code128(uint32_t amax) {
    const int E = (int)(amax >> 23);
    if (E == 255) return 255u;
    const int s = E - 135 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(max(s, -127) + 127);  // s <= 120: no upper clamp is reached
}

// 2^-s for a code below 255: s in [-127, 120].
__device__ __forceinline__ uint32_t inv_scale128(uint32_t code) { return (254u - code) << 23; }

template <Elt ELT>
__device__ __forceinline__ uint32_t load_f32(const void* x, int64_t i) {
    if constexpr (ELT == Elt::BF16) return (uint32_t)static_cast<const uint16_t*>(x)[i] << 16;
    return static_cast<const uint32_t*>(x)[i];
}

template <Elt ELT>
__host__ __device__ constexpr int64_t elt_bytes() {
    return ELT == Elt::BF16 ? 2 : 4;
}

// A word of one fp32 or two bf16 elements, NaN made canonical.
template <Elt ELT>
__device__ __forceinline__ uint32_t canonical_word(uint32_t v) {
    if constexpr (ELT == Elt::BF16) {
        if ((v & 0x7FFFu) > 0x7F80u) v = (v & 0xFFFF0000u) | 0x7FC0u;
        if ((v & 0x7FFFFFFFu) > 0x7F80FFFFu) v = (v & 0xFFFFu) | 0x7FC00000u;
    } else if ((v & 0x7FFFFFFFu) > 0x7F800000u) {
        v = 0x7FC00000u;
    }
    return v;
}

// 16 consecutive elements as fp32 patterns, 32-byte loads.
template <Elt ELT>
struct Unit {
    uint32_t w[ELT == Elt::BF16 ? 8 : 16];

    __device__ __forceinline__ void load(const void* x, int64_t i) {
        if constexpr (ELT == Elt::BF16) {
            ld32(w, static_cast<const uint16_t*>(x) + i);
        } else {
            ld32(reinterpret_cast<uint32_t(&)[8]>(w[0]), static_cast<const uint32_t*>(x) + i);
            ld32(reinterpret_cast<uint32_t(&)[8]>(w[8]), static_cast<const uint32_t*>(x) + i + 8);
        }
    }
    // The same from what every row reads (a norm's weight): kept in L1.
    __device__ __forceinline__ void load_shared(const void* x, int64_t i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + i * elt_bytes<ELT>());
#pragma unroll
        for (int q = 0; q < (ELT == Elt::BF16 ? 2 : 4); ++q) {
            const uint4 v = __ldg(p + q);
            w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
        }
    }
    __device__ __forceinline__ void store(void* x, int64_t i) const {
        char* p = static_cast<char*>(x) + i * elt_bytes<ELT>();
        st32(p, reinterpret_cast<const uint32_t(&)[8]>(w[0]));
        if constexpr (ELT == Elt::FP32) st32(p + 32, reinterpret_cast<const uint32_t(&)[8]>(w[8]));
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& v : w) v = 0;
    }
    __device__ __forceinline__ uint32_t at(int i) const {
        if constexpr (ELT == Elt::BF16) return i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16;
        return w[i];
    }
    __device__ __forceinline__ float f(int i) const { return __uint_as_float(at(i)); }
    __device__ __forceinline__ float2 f2(int j) const { return make_float2(f(2 * j), f(2 * j + 1)); }
    // Rounds values 2j and 2j + 1; NaN is left as the conversion makes it.
    __device__ __forceinline__ void set2(int j, float lo, float hi) {
        if constexpr (ELT == Elt::BF16) {
            w[j] = bf16x2_from_f32(hi, lo);
        } else {
            w[2 * j] = __float_as_uint(lo);
            w[2 * j + 1] = __float_as_uint(hi);
        }
    }
    // Adds, each sum rounded once.
    __device__ __forceinline__ void add(const Unit& o) {
        if constexpr (ELT == Elt::BF16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = bf2_add(w[j], o.w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = f32_add(w[j], o.w[j]);
        }
    }
    // NaN elements to the canonical NaN.
    __device__ __forceinline__ void canonical() {
#pragma unroll
        for (uint32_t& v : w) v = canonical_word<ELT>(v);
    }
};

// One element, rounded to nearest even; NaN comes out canonical.
template <Elt ELT>
__device__ __forceinline__ void store_f32(void* p, int64_t i, float v) {
    const bool nan = (__float_as_uint(v) & 0x7FFFFFFFu) > 0x7F800000u;
    if constexpr (ELT == Elt::BF16) static_cast<uint16_t*>(p)[i] = nan ? 0x7FC0 : (uint16_t)bf16x2_from_f32(0.0f, v);
    else static_cast<uint32_t*>(p)[i] = nan ? 0x7FC00000u : __float_as_uint(v);
}

__device__ __forceinline__ uint8_t e4m3_byte(float v, uint32_t code) {
    return code == 255u ? 0x7F : (uint8_t)e4m3x2_from_f32(0u, f32_mul(__float_as_uint(v), inv_scale128(code)));
}

// 16 bytes into shared memory, asynchronously; past L1.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// Two floats in one 64-bit register: one instruction for both.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float ex2_approx(float t) {
    float p;
    asm("ex2.approx.f32 %0, %1;" : "=f"(p) : "f"(t));
    return p;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
    return a;
}

// exp(-a) for a >= 0, off by 3e-7 of itself at most.  exp(-a) = 2^t with
// t = -a log2(e); the product is kept to twice its bits, t + r, so that its
// rounding does not grow with a, and 2^(t + r) = 2^t (1 + r ln 2) for the
// small r.  a is cut off at 160, where the result is zero either way.  NaN stays
// NaN.
constexpr float kExpHi = -1.4426950216293335f, kExpLo = -1.9259629911e-8f, kLn2 = 0.6931471805599453f, kExpEnd = 160.0f;
__device__ __forceinline__ float exp_neg(float a) {
    a = min_nan(a, kExpEnd);
    const float t = fmul(a, kExpHi), r = ffma(a, kExpLo, ffma(a, kExpHi, -t)), p = ex2_approx(t);
    return ffma(fmul(p, kLn2), r, p);
}
__device__ __forceinline__ float rcp_approx(float v) {
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v));
    return v;
}

// s = 1 / (1 + exp(-x)) and 1 - s, each to a few units in its last place at
// either end: the exponential is that of -|x|, the sum lies in [1, 2].
struct Sigmoid {
    float s, rest;
    __device__ __forceinline__ explicit Sigmoid(float x) {
        const float e = exp_neg(fabsf(x)), inv = rcp_approx(fadd(1.0f, e)), low = fmul(e, inv);
        const bool neg = (int32_t)__float_as_uint(x) < 0;
        s = neg ? low : inv;
        rest = neg ? inv : low;
    }
};

// Largest magnitude of `m` and two more values; NaN if one of them is.
__device__ __forceinline__ float absmax3(float m, float a, float b) {
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(a), "f"(b));
    return m;
}

// 16 E4M3 payloads of a block with scale code `code`.
__device__ __forceinline__ void e4m3_store16(uint8_t* p, const float (&v)[16], uint32_t code) {
    const float2 inv = both(__uint_as_float(inv_scale128(code)));
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 lo = mul2(make_float2(v[4 * j], v[4 * j + 1]), inv), hi = mul2(make_float2(v[4 * j + 2], v[4 * j + 3]), inv);
        o[j] = e4m3x2_from_f32(__float_as_uint(lo.y), __float_as_uint(lo.x)) | e4m3x2_from_f32(__float_as_uint(hi.y), __float_as_uint(hi.x)) << 16;
        if (code == 255u) o[j] = 0x7F7F7F7Fu;
    }
    st16(p, o[0], o[1], o[2], o[3]);
}

inline bool on_bytes(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Rows of units: the first element and the stride on 32 bytes.
template <Elt ELT>
bool unit_rows(const void* p, int64_t rows, int64_t ld) {
    return on_bytes(p, 32) && (rows <= 1 || ld * elt_bytes<ELT>() % 32 == 0);
}

}  // namespace mxq
