// kernel_glr.cuh -- the gated linear recurrence, one thread per channel.
//
//   s_t = sigmoid(gate_t),  u_t = sigmoid(input_gate_t) x_t  (or x_t)
//   no rate: a_t = s_t, beta_t = 1 - s_t;   rate c: a_t = exp(-c s_t), beta_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + beta_t u_t,  y_t = h_t
//
// Each thread walks its channel token by token with the state in a register: no
// exchange between threads, so this is the form for a few tokens (a decode step), where
// the batch's channels alone fill the device.
#pragma once

#include "device_utils.cuh"
#include "glr_math.cuh"

namespace sscan {
namespace glr {

constexpr int kRun = 8;  // tokens between two saved states

struct FwdParams {
    const void *x, *gate, *igate;
    const float *rate, *h0;
    void *y;
    float *h_final, *states;
    int64_t B, L, D, nruns;
};

struct BwdParams {
    const void *x, *gate, *igate, *dy;
    const float *rate, *states, *dh_final;
    void *dx, *dgate, *digate;
    float *dh0, *part;  // part: [parts][D] partial sums of drate (with a rate)
    int64_t B, L, D, nruns;
};

// One token's decay and input: a, b = beta u
template <bool DECAY, bool IG>
__device__ __forceinline__ void token(float x, float g, float ig, float c, float &a, float &b) {
    float s, n, beta;
    sigmoid_pair(g, s, n);
    if constexpr (DECAY) {
        float m;
        decay(c * s, a, m);
        beta = sqrt_approx(m * (2.0f - m));
    } else {
        a = s;
        beta = n;
    }
    if constexpr (IG) {
        float si, ni;
        sigmoid_pair(ig, si, ni);
        x *= si;
    }
    b = beta * x;
}

// One token's factors of the gradients, given the state before it: with G the whole
// gradient of h_t,  dx = G px,  dig = G pi,  dgate = G pg,  drate += G pr.
//   dh/da = h' + u dbeta/da;  no rate: dbeta/da = -1, da/dg = s n
//   rate: dbeta/da = -a/beta, da/dz = -a, dz/dg = c s n, dz/dc = s.
// a/beta diverges as z -> 0 but s a^2/beta -> 0 with it: 1/beta is taken of at least
// 2^-126, which keeps every product finite and its limit 0.
template <bool DECAY, bool IG>
__device__ __forceinline__ void token_grad(float x, float g, float ig, float c, float hp, float &a, float &b,
                                           float &px, float &pi, float &pg, float &pr) {
    float s, n, beta;
    sigmoid_pair(g, s, n);
    float si = 1.0f, ni = 0.0f, u = x;
    if constexpr (IG) {
        sigmoid_pair(ig, si, ni);
        u = x * si;
    }
    if constexpr (DECAY) {
        float m;
        decay(c * s, a, m);
        const float w = m * (2.0f - m);
        const float ib = rsqrt_approx(fmaxf(w, 1.17549435e-38f));
        beta = w * ib;
        const float q = -s * (a * (hp - a * ib * u));  // dh/dc
        pr = q;
        pg = q * (c * n);
    } else {
        a = s;
        beta = n;
        pr = 0.0f;
        pg = (hp - u) * (s * n);
    }
    b = beta * u;
    px = beta * si;
    pi = IG ? b * ni : 0.0f;
}

constexpr int kStepThreads = 128;

template <class IO, bool DECAY, bool IG>
__global__ void __launch_bounds__(kStepThreads) glr_step_kernel(const FwdParams p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i - b * p.D;
    const IO *x = static_cast<const IO *>(p.x), *g = static_cast<const IO *>(p.gate), *ig = static_cast<const IO *>(p.igate);
    IO *y = static_cast<IO *>(p.y);
    const float c = DECAY ? p.rate[d] : 0.0f;
    float h = p.h0 ? p.h0[i] : 0.0f;
    for (int64_t t = 0; t < p.L; ++t) {
        const int64_t at = (b * p.L + t) * p.D + d;
        if (p.states && t % kRun == 0) p.states[(b * p.nruns + t / kRun) * p.D + d] = h;
        float a, in;
        token<DECAY, IG>(Io<IO>::widen(Io<IO>::ld(x + at)), Io<IO>::widen(Io<IO>::ld(g + at)),
                         IG ? Io<IO>::widen(Io<IO>::ld(ig + at)) : 0.0f, c, a, in);
        h = fmaf(a, h, in);
        Io<IO>::st(y + at, h);
    }
    if (p.h_final) p.h_final[i] = h;
}

template <class IO, bool DECAY, bool IG>
__global__ void __launch_bounds__(kStepThreads) glr_step_backward_kernel(const BwdParams p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i - b * p.D;
    const IO *x = static_cast<const IO *>(p.x), *g = static_cast<const IO *>(p.gate), *ig = static_cast<const IO *>(p.igate);
    const IO *dy = static_cast<const IO *>(p.dy);
    const float c = DECAY ? p.rate[d] : 0.0f;
    float e = p.dh_final ? p.dh_final[i] : 0.0f, dc = 0.0f;
    for (int64_t run = p.nruns - 1; run >= 0; --run) {
        float a[kRun], px[kRun], pi[kRun], pg[kRun], pr[kRun];
        float h = p.states[(b * p.nruns + run) * p.D + d];
        const int64_t t0 = run * kRun;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (t0 + k >= p.L) break;
            const int64_t at = (b * p.L + t0 + k) * p.D + d;
            float in;
            token_grad<DECAY, IG>(Io<IO>::widen(Io<IO>::ld(x + at)), Io<IO>::widen(Io<IO>::ld(g + at)),
                                  IG ? Io<IO>::widen(Io<IO>::ld(ig + at)) : 0.0f, c, h, a[k], in, px[k], pi[k], pg[k],
                                  pr[k]);
            h = fmaf(a[k], h, in);
        }
#pragma unroll
        for (int k = kRun - 1; k >= 0; --k) {
            if (t0 + k >= p.L) continue;
            const int64_t at = (b * p.L + t0 + k) * p.D + d;
            const float G = Io<IO>::widen(Io<IO>::ld(dy + at)) + e;
            e = a[k] * G;
            Io<IO>::st(static_cast<IO *>(p.dx) + at, G * px[k]);
            Io<IO>::st(static_cast<IO *>(p.dgate) + at, G * pg[k]);
            if constexpr (IG) Io<IO>::st(static_cast<IO *>(p.digate) + at, G * pi[k]);
            if constexpr (DECAY) dc = fmaf(G, pr[k], dc);
        }
    }
    if (p.dh0) p.dh0[i] = e;
    if constexpr (DECAY) p.part[i] = dc;
}

}  // namespace glr
}  // namespace sscan
