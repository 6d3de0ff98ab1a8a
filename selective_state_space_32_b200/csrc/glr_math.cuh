// glr_math.cuh -- the gate arithmetic of the gated linear recurrence, one token of one
// channel, in fp32.
//
// s = sigmoid(g) and its complement n = 1 - s come from t = e^-|g| <= 1: one of them is
// 1/(1 + t), the other t/(1 + t), so neither cancels nor overflows (g = +-inf gives 1
// and 0).  Without a rate the decay is a = s and the input factor beta = n.  With a
// rate c, a = e^-z, z = c s, and beta = sqrt(1 - a^2) = sqrt(m (2 - m)) with
// m = 1 - a.  m cancels when z is small, where a long memory lives, so there
// (z <= 1/8) m = z phi(-z), phi(z) = (e^z - 1)/z by the polynomial psi2 (3.3e-7
// relative), and a = 1 - m (correctly rounded up to that: the error of a slow decay
// is not the MUFU's 2^-22 times the horizon 1/(1 - a)); beyond, a = 2^(-z log2 e) on
// the MUFU and m = 1 - a >= 0.117.
#pragma once

#include "device_utils.cuh"

namespace sscan {
namespace glr {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// s = sigmoid(g), n = 1 - s
__device__ __forceinline__ void sigmoid_pair(float g, float &s, float &n) {
    const float t = ex2(-fabsf(g) * kLog2e);
    const float big = rcp(1.0f + t), small = t * big;
    s = g >= 0.0f ? big : small;
    n = g >= 0.0f ? small : big;
}

// a = e^-z and m = 1 - a for z = c s >= 0 (c in nats)
__device__ __forceinline__ void decay(float z, float &a, float &m) {
    const float e = z * kLog2e;
    float q = fmaf(-1.387602649629116e-02f, e, 8.013805747032166e-02f);  // psi2 at -e, scalar
    q = fmaf(q, -e, 3.4657374024391174e-01f);
    q = fmaf(q, -e, 9.999997615814209e-01f);
    const float ms = z * q;
    const float al = ex2(-e);
    const bool slow = z <= 0.125f;
    m = slow ? ms : 1.0f - al;
    a = slow ? 1.0f - ms : al;
}

}  // namespace glr
}  // namespace sscan
