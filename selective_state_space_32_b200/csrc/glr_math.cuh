// glr_math.cuh -- the gate arithmetic of the gated linear recurrence in fp32, two values
// at a time (two channels of a token, or two tokens of a channel) as packed pairs: the
// kernels are near their issue rate, and a packed operation takes one slot for two values.
//
// sigmoid(g) = 1 / (1 + E), E = e^-g: accurate relative to its size for every g, since
// nothing cancels (E overflowing gives 0).  Its complement is E sigmoid(g), with E's
// exponent held below 126 so that the product stays finite.
//
// A rate c gives the decay a = e^-z, z = c s, and beta = sqrt(1 - a^2) = sqrt(m (2 - m))
// with m = 1 - a.  m must keep its digits when z is small, where a long memory lives, so
// both come from one range reduction: e = z log2 e = j + f with j = round(e),
// p = 2^-f - 1 = f times a polynomial (no constant term: relative accuracy at f -> 0),
// S = 2^-j, a = S + S p and m = (1 - S) - S p, which is -p itself when j = 0.  It runs on
// the FMA pipe: the MUFU has 16 lanes an SM and clock, and with the sigmoids and the
// square root the exponential would make it the bound.
#pragma once

#include "device_utils.cuh"

namespace sscan {
namespace glr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// min that keeps NaN
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
template <class F>
__device__ __forceinline__ f2 map2(f2 v, F f) {
    float a, b;
    unpack2(v, a, b);
    return pack2(f(a), f(b));
}

// 1 + e^-g
__device__ __forceinline__ f2 one_plus_exp(f2 g) {
    return add2(map2(mul2(g, splat2(-kLog2e)), [](float e) { return ex2(e); }), splat2(1.0f));
}
__device__ __forceinline__ f2 rcp2(f2 v) {
    return map2(v, [](float x) { return rcp(x); });
}
// s = sigmoid(g), n = 1 - s
__device__ __forceinline__ void sigmoid2(f2 g, f2 &s, f2 &n) {
    const f2 E = map2(mul2(g, splat2(-kLog2e)), [](float e) { return ex2(min_nan(e, 126.0f)); });
    s = rcp2(add2(E, splat2(1.0f)));
    n = mul2(E, s);
}

// a - v on the FMA pipe (flipping the sign bits would be two integer operations)
__device__ __forceinline__ f2 minus2(f2 a, f2 v) { return fma2(v, splat2(-1.0f), a); }

// Rates above 2^21, infinity among them, act as 2^21: e below stays under 2^22, where its
// rounding is exact.  At every gate above -9.9 they decay by less than 2^-126 either way.
constexpr float kMaxRate = 2097152.0f;
__device__ __forceinline__ f2 capped_rate(f2 c) {
    return map2(c, [](float v) { return min_nan(v, kMaxRate); });
}

// a = e^-z and m = 1 - a, z = s c, from s in [0, 1] and cl = c log2 e.  j is held at 126, so that
// decays below 2^-126 are about 2^-126.  (Held in t, which only S waits for: 1 x 131072 x 2048
// bf16 606 us, without a hold 602; held in e, which f waits for too, 632.)
// 2^-f - 1 = f q(f), with -q(-f) = ln 2 times the degree-5 minimax polynomial of (e^z - 1)/z
// on |f| <= 1/2 (csrc/gen_phi_poly.py 5 0.3465735902799726 --log2: 1.1e-8, 1.4e-7 evaluated
// in fp32).
__device__ __forceinline__ void decay2(f2 s, f2 cl, f2 &a, f2 &m) {
    const f2 kShift = splat2(12582912.0f);  // 1.5 * 2^23
    const f2 t = fma2(s, cl, kShift);       // j in the low mantissa bits
    const f2 f = fma2(s, cl, minus2(kShift, t));  // e - j
    f2 q = fma2(splat2(1.5403512225020677e-04f), f, splat2(-1.3390735257416964e-03f));
    q = fma2(q, f, splat2(9.6182376146316528e-03f));
    q = fma2(q, f, splat2(-5.5503576993942261e-02f));
    q = fma2(q, f, splat2(2.4022650718688965e-01f));
    q = fma2(q, f, splat2(-6.9314718246459961e-01f));
    const f2 p = mul2(q, f);
    float t0, t1;
    unpack2(map2(t, [](float v) { return min_nan(v, 12582912.0f + 126.0f); }), t0, t1);
    const f2 S = pack2(__uint_as_float(__float_as_uint(t0) * 0xff800000u + 0x3f800000u),  // 2^-j
                       __uint_as_float(__float_as_uint(t1) * 0xff800000u + 0x3f800000u));
    a = fma2(S, p, S);
    m = fma2(S, mul2(p, splat2(-1.0f)), minus2(splat2(1.0f), S));
}

// Two tokens' or channels' decay a and input b = beta sigmoid(ig) x.  cl: rate log2 e.
template <bool DECAY, bool IG>
__device__ __forceinline__ void token2(f2 x, f2 g, f2 ig, f2 cl, f2 &a, f2 &b) {
    if constexpr (DECAY) {
        f2 m;
        decay2(rcp2(one_plus_exp(g)), cl, a, m);
        const f2 r = minus2(splat2(2.0f), m), w = mul2(m, r);
        f2 v = fma2(m, r, splat2(kTiny));  // w = 0 (a = 1) gives beta = 0, not 0 * inf
        // beta sigmoid(ig) = sqrt(w) / (1 + E) = w rsqrt(w q^2) k with q = (1 + E) k: one MUFU operation
        // for the square root and the quotient.  k is the power of two, from the complement of
        // 1 + E's exponent, that puts q in [2, 4).  (Without k the square overflows for ig below -44; a
        // reciprocal of its own: 1 x 131072 x 2048 bf16 632 us instead of 602.  k into x, which
        // overflows where x is above half the largest number: 591.)
        f2 k = 0;
        if constexpr (IG) {
            f2 q = add2(map2(mul2(ig, splat2(-kLog2e)), [](float e) { return ex2(min_nan(e, 126.0f)); }), splat2(1.0f));
            k = map2(q, [](float y) { return __uint_as_float(~__float_as_uint(y) & 0x7f800000u); });
            q = mul2(q, k);
            v = mul2(v, mul2(q, q));
        }
        f2 f = mul2(w, map2(v, [](float y) { return rsqrt_approx(y); }));
        if constexpr (IG) f = mul2(f, k);
        b = mul2(f, x);
    } else {
        f2 n;
        sigmoid2(g, a, n);
        if constexpr (IG) x = mul2(x, rcp2(one_plus_exp(ig)));
        b = mul2(n, x);
    }
}

// Two tokens' or channels' factors of the gradients that need no state: with G the whole
// gradient of h_t,  dx = G px,  dig = G pi,  dgate = G kg (v - h_{t-1}),
// drate += G kr (v - h_{t-1}):
//   dh/da = h_{t-1} + u dbeta/da;  no rate: dbeta/da = -1, da/dg = s n: v = u, kg = -s n
//   rate: dbeta/da = -a/beta, da/dz = -a, dz/dc = s, dz/dg = c s n: v = a u / beta,
//   kr = s a, kg = kr c n.
// a/beta diverges as z -> 0, but s a^2/beta -> 0 with it: 1/beta is taken of at least
// 2^-126, which keeps every product finite and its limit 0.
template <bool DECAY, bool IG>
__device__ __forceinline__ void token_grad2(f2 x, f2 g, f2 ig, f2 c, f2 cl, f2 &a, f2 &b, f2 &v, f2 &px, f2 &pi, f2 &kg,
                                            f2 &kr) {
    f2 s, n, si = 0, ni = 0, u = x, beta;
    sigmoid2(g, s, n);
    if constexpr (IG) {
        sigmoid2(ig, si, ni);
        u = mul2(x, si);
    }
    if constexpr (DECAY) {
        f2 m;
        decay2(s, cl, a, m);
        const f2 r = minus2(splat2(2.0f), m), w = mul2(m, r);
        const f2 ib = map2(fma2(m, r, splat2(kTiny)), [](float y) { return rsqrt_approx(y); });
        beta = mul2(w, ib);
        v = mul2(mul2(a, ib), u);
        kr = mul2(s, a);
        kg = mul2(kr, mul2(c, n));
    } else {
        a = s;
        beta = n;
        v = u;
        kr = 0;
        kg = mul2(mul2(s, splat2(-1.0f)), n);
    }
    b = mul2(beta, u);
    px = IG ? mul2(beta, si) : beta;
    pi = IG ? mul2(b, ni) : 0;
}

}  // namespace glr
}  // namespace sscan
