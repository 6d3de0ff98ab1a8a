// kernel_norm.cuh -- layer norm over the last axis of [rows, D], forward and backward,
// with the residual addition in front of it.
//
//   s = x + residual, rounded to the residual's type (no residual: s = x)
//   mu = mean(s) (0 with RMS), rstd = 1 / sqrt(mean((s - mu)^2) + eps), z = (s - mu) rstd
//   y = z w + b
//   ds = rstd (w dy - mean(w dy) - z mean(w dy z)) + dresidual   (RMS: without mean(w dy))
//   dw = sum over rows of dy z,  db = sum over rows of dy
//
// Statistics are of the rounded s, the value that the residual stream holds and that the
// backward pass reads; they are taken in two passes (mean, then the centred squares) in
// fp32, so that a mean far from zero costs no digits of the variance.
#pragma once

#include "device_utils.cuh"

namespace sscan {
namespace norm {

constexpr int kRowThreads = 256;

struct FwdParams {
    const void *x, *residual;
    const float *weight, *bias;
    void *y, *residual_out;
    float *mean, *rstd;
    int64_t rows, D;
    float eps;
};

struct BwdParams {
    const void *dy, *s, *dresidual;
    const float *mean, *rstd, *weight;
    void *ds, *dx;  // ds in s's type; dx in dy's type (null: the same type, ds serves)
    float *part;    // [2][parts][D]: dw, db of each block's rows
    int64_t rows, D;
    int want_dw, want_db;
};

__device__ __forceinline__ float rsqrt_fp32(float v) { return 1.0f / sqrtf(v); }

// Sum over the block's 256 threads, the same value in every thread (sm: 8 floats; the
// caller's next use of the same sm comes after another barrier of its own).
__device__ __forceinline__ float block_sum(float v, float *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kRowThreads / 32; ++k) s += sm[k];
    __syncthreads();
    return s;
}

template <class IO, class R, bool RES>
__device__ __forceinline__ float load_sum(const IO *x, const R *r, int64_t i) {
    const float v = Io<IO>::widen(Io<IO>::ld(x + i));
    if constexpr (!RES) return v;
    R q;
    Io<R>::st(&q, v + Io<R>::widen(Io<R>::ld(r + i)));
    return Io<R>::widen(q);
}

// IO: x, y; R: residual and residual_out.  One block per row, any D.
template <class IO, class R, bool RES, bool RMS>
__global__ void __launch_bounds__(kRowThreads) norm_forward_kernel(const FwdParams p) {
    __shared__ float sm[kRowThreads / 32];
    const float inv_d = 1.0f / static_cast<float>(p.D);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const IO *x = static_cast<const IO *>(p.x) + row * p.D;
        const R *r = RES ? static_cast<const R *>(p.residual) + row * p.D : nullptr;
        float mu = 0.0f;
        if (RES || !RMS) {
            float v = 0.0f;
            for (int64_t i = threadIdx.x; i < p.D; i += kRowThreads) {
                const float s = load_sum<IO, R, RES>(x, r, i);
                if constexpr (RES) Io<R>::st(static_cast<R *>(p.residual_out) + row * p.D + i, s);
                v += s;
            }
            if constexpr (!RMS) mu = block_sum(v, sm) * inv_d;
        }
        float v = 0.0f;
        for (int64_t i = threadIdx.x; i < p.D; i += kRowThreads) {
            const float s = load_sum<IO, R, RES>(x, r, i) - mu;
            v = fmaf(s, s, v);
        }
        const float rstd = rsqrt_fp32(block_sum(v, sm) * inv_d + p.eps);
        for (int64_t i = threadIdx.x; i < p.D; i += kRowThreads) {
            float o = (load_sum<IO, R, RES>(x, r, i) - mu) * rstd;
            if (p.weight) o *= __ldg(p.weight + i);
            if (p.bias) o += __ldg(p.bias + i);
            Io<IO>::st(static_cast<IO *>(p.y) + row * p.D + i, o);
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mu;
            if (p.rstd) p.rstd[row] = rstd;
        }
    }
}

// IO: dy, dx; R: s, dresidual, ds.  Block k takes rows k, k + gridDim.x, ... and keeps its
// columns' dw and db in its own rows of part (each entry touched by one thread only).
template <class IO, class R, bool RMS>
__global__ void __launch_bounds__(kRowThreads) norm_backward_kernel(const BwdParams p) {
    __shared__ float sm[kRowThreads / 32];
    const float inv_d = 1.0f / static_cast<float>(p.D);
    float *pw = p.part + blockIdx.x * p.D, *pb = p.part + (gridDim.x + blockIdx.x) * p.D;
    bool first = true;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const IO *dy = static_cast<const IO *>(p.dy) + row * p.D;
        const R *s = static_cast<const R *>(p.s) + row * p.D;
        const float mu = RMS ? 0.0f : p.mean[row], rstd = p.rstd[row];
        float v1 = 0.0f, v2 = 0.0f;
        for (int64_t i = threadIdx.x; i < p.D; i += kRowThreads) {
            const float z = (Io<R>::widen(Io<R>::ld(s + i)) - mu) * rstd;
            float w = Io<IO>::widen(Io<IO>::ld(dy + i));
            if (p.weight) w *= __ldg(p.weight + i);
            v1 += w;
            v2 = fmaf(w, z, v2);
        }
        const float m1 = RMS ? 0.0f : block_sum(v1, sm) * inv_d;
        const float m2 = block_sum(v2, sm) * inv_d;
        for (int64_t i = threadIdx.x; i < p.D; i += kRowThreads) {
            const float z = (Io<R>::widen(Io<R>::ld(s + i)) - mu) * rstd;
            const float g = Io<IO>::widen(Io<IO>::ld(dy + i));
            const float w = p.weight ? g * __ldg(p.weight + i) : g;
            float o = rstd * (w - m1 - z * m2);
            if (p.dresidual) o += Io<R>::widen(Io<R>::ld(static_cast<const R *>(p.dresidual) + row * p.D + i));
            Io<R>::st(static_cast<R *>(p.ds) + row * p.D + i, o);
            if (p.dx) Io<IO>::st(static_cast<IO *>(p.dx) + row * p.D + i, o);
            if (p.want_dw) pw[i] = first ? g * z : fmaf(g, z, pw[i]);
            if (p.want_db) pb[i] = first ? g : g + pb[i];
        }
        first = false;
    }
}

}  // namespace norm
}  // namespace sscan
