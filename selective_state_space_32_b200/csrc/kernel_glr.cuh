// kernel_glr.cuh -- the gated linear recurrence, one thread per channel or channel pair.
//
//   s_t = sigmoid(gate_t),  u_t = sigmoid(input_gate_t) x_t  (or x_t)
//   no rate: a_t = s_t, beta_t = 1 - s_t;   rate c: a_t = exp(-c s_t), beta_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + beta_t u_t,  y_t = h_t
//
// Each thread walks its channels token by token with the state in a register: no
// exchange between threads, so this is the form for a few tokens (a decode step), where
// the batch's channels alone fill the device.  Measured on B200: 1 row of 2048 channels 2.3 us,
// 256 rows 3.3 us (10.5 MB: 1.6 us at the copy rate; launch and one memory latency the rest).
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
    float *dh0, *part;  // part: partial sums of drate (with a rate), rows of D
    int64_t B, L, D, nruns;
};

// V = 1 or 2 consecutive channels as a pair (V = 1: the second half repeats the first)
template <class IO, int V>
__device__ __forceinline__ f2 load_channels(const IO *p) {
    if constexpr (V == 1) {
        return splat2(Io<IO>::widen(Io<IO>::ld(p)));
    } else if constexpr (sizeof(IO) == 4) {
        const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
        return pack2(v.x, v.y);
    } else {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(p));
        return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}
template <class IO, int V>
__device__ __forceinline__ void store_channels(IO *p, f2 v) {
    float a, b;
    unpack2(v, a, b);
    if constexpr (V == 1) {
        Io<IO>::st(p, a);
    } else if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<float2 *>(p) = make_float2(a, b);
    } else {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
        *reinterpret_cast<uint32_t *>(p) = w;
    }
}

constexpr int kStepThreads = 128;

// V = 2 wants an even D.  The plain (not read-only) load of h0 matters: h_final may be h0.
template <class IO, int V, bool DECAY, bool IG>
__global__ void __launch_bounds__(kStepThreads) glr_step_kernel(const FwdParams p) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * kStepThreads + threadIdx.x) * V;
    if (i >= p.B * p.D) return;
    const int64_t b = i / p.D, d = i - b * p.D;
    const int64_t row0 = b * p.L * p.D + d;
    const IO *x = static_cast<const IO *>(p.x) + row0, *g = static_cast<const IO *>(p.gate) + row0;
    const IO *ig = static_cast<const IO *>(p.igate) + (IG ? row0 : 0);
    IO *y = static_cast<IO *>(p.y) + row0;
    f2 h = 0, cl = 0;
    if (p.h0) h = V == 2 ? pack2(p.h0[i], p.h0[i + V - 1]) : splat2(p.h0[i]);
    if constexpr (DECAY) cl = mul2(capped_rate(load_channels<float, V>(p.rate + d)), splat2(kLog2e));
    for (int64_t t = 0; t < p.L; ++t) {
        if (p.states && t % kRun == 0)
            store_channels<float, V>(p.states + (b * p.nruns + t / kRun) * p.D + d, h);
        f2 a, in;
        token2<DECAY, IG>(load_channels<IO, V>(x + t * p.D), load_channels<IO, V>(g + t * p.D),
                          IG ? load_channels<IO, V>(ig + t * p.D) : 0, cl, a, in);
        h = fma2(a, h, in);
        store_channels<IO, V>(y + t * p.D, h);
    }
    if (p.h_final) store_channels<float, V>(p.h_final + i, h);
}

}  // namespace glr
}  // namespace sscan
