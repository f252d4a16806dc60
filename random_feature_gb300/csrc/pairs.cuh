// Two floats at a time: packed arithmetic, and the gates in it.
#pragma once

#include "ssm_internal.h"

namespace favor {

// Two floats in one register pair (pack2 and its kin): one instruction for both.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) : v(pack2(x, y)) {}
    __device__ __forceinline__ explicit F2(uint64_t u) : v(u) {}
    __device__ __forceinline__ float x() const { float a, b; unpack2(v, a, b); return a; }
    __device__ __forceinline__ float y() const { float a, b; unpack2(v, a, b); return b; }
};
__device__ __forceinline__ F2 both(float x) { return F2(x, x); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) { return F2(mul2(a.v, b.v)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return F2(fma2(a.v, b.v, c.v)); }
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
template <typename F>
__device__ __forceinline__ F2 each(F2 a, F f) { return F2(f(a.x()), f(a.y())); }

// ------------------------------------------------------------------ gates
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What sigmoid2 adds to x, from a bias.
template <typename T>
__device__ __forceinline__ F2 sigmoid_bias(F2 b) { return sizeof(T) == 2 ? b * both(-kLog2e) : b; }
// sigmoid(x + bias).  16-bit storage: one product and one sum make the exponent, and the approximate forms follow;
// the relative error is under 2^-18 for |x|, |bias| < 16 (two roundings of an exponent of up to 46, 3 2^-20 in it).
// fp32: sigmoids.
template <typename T>
__device__ __forceinline__ F2 sigmoid2(F2 x, F2 bias) {
    if (sizeof(T) == 2) {
        const F2 e(ex2_2(fma2(x, both(-kLog2e), bias).v));
        return each(e + both(1.f), [](float d) { return rcp_approx(d); });
    }
    return each(x + bias, [](float v) { float s, n; sigmoids<T>(v, s, n); return s; });
}
// sigmoid(x) and sigmoid(-x) = e sigmoid(x), e = e^-x, which is kept finite for it (but a NaN, a NaN).  sigmoid(x)
// itself is 0 from there on, as a product with an x of the type's lowest value has to be (2^-126 makes -4 of bf16's).
// KEPT: 2^-126 stays, for a decay, whose state is nowhere near 2^126 (the recurrence without rates takes 3% longer
// with the 0).
template <typename T, bool KEPT = false>
__device__ __forceinline__ void sigmoids2(F2 x, F2 bias, F2& s, F2& sn) {
    if (sizeof(T) == 2) {
        const F2 t = each(fma2(x, both(-kLog2e), bias), [](float v) {
            float m;
            asm("min.NaN.f32 %0, %1, 0f42FC0000;" : "=f"(m) : "f"(v));      // 126
            return m;
        });
        const F2 e(ex2_2(t.v)), r = each(e + both(1.f), [](float d) { return rcp_approx(d); });
        sn = e * r;
        s = KEPT ? r : F2(t.x() >= 126.f ? 0.f : r.x(), t.y() >= 126.f ? 0.f : r.y());
        return;
    }
    const F2 raw = x + bias;
    float s0, n0, s1, n1;
    sigmoids<T>(raw.x(), s0, n0);
    sigmoids<T>(raw.y(), s1, n1);
    s = F2(s0, s1);
    sn = F2(n0, n1);
}
template <typename T>
__device__ __forceinline__ F2 silu2(F2 x) {
    if (sizeof(T) == 2)
        return x * each(F2(ex2_2((x * both(-kLog2e)).v)) + both(1.f), [](float d) { return rcp_approx(d); });
    return x * sigmoid2<T>(x, both(0.f));
}

__device__ __forceinline__ F2 to_f2(uint32_t u) {
    return F2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t from_f2(F2 x, __nv_bfloat16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x(), x.y());
    return *reinterpret_cast<const uint32_t*>(&a);
}
__device__ __forceinline__ float2 from_f2(F2 x, float) { return make_float2(x.x(), x.y()); }

}  // namespace favor
