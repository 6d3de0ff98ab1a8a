// glr.cu -- C ABI of the gated linear recurrence (kernels in kernel_glr.cuh): argument
// checks, the choice of the kernel and the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "abi_checks.cuh"
#include "column_sums.cuh"
#include "kernel_glr.cuh"
#include "sscan.h"

using namespace sscan;

namespace {

// Sizes that every index and grid of the kernels can hold.
int check_sizes(int64_t B, int64_t L, int64_t D, int dtype) {
    if (B < 1 || D < 1 || L < 0) return SSCAN_ERR_INVALID;
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    const int64_t kMax = int64_t(1) << 31;
    if (B >= kMax || D >= kMax || B * D >= kMax * 16) return SSCAN_ERR_UNSUPPORTED;
    if (L > (int64_t(1) << 40) || (L > 0 && B * D > (int64_t(1) << 48) / L)) return SSCAN_ERR_UNSUPPORTED;
    return SSCAN_OK;
}

int64_t runs(int64_t L) { return ceil_div(L, glr::kRun); }

template <class IO, bool DECAY, bool IG>
int launch_forward(const glr::FwdParams &p, cudaStream_t s) {
    const int64_t blocks = ceil_div(p.B * p.D, glr::kStepThreads);
    glr::glr_step_kernel<IO, DECAY, IG><<<static_cast<unsigned>(blocks), glr::kStepThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

template <class IO, bool DECAY, bool IG>
int launch_backward(const glr::BwdParams &p, float *drate, cudaStream_t s) {
    const int64_t blocks = ceil_div(p.B * p.D, glr::kStepThreads);
    glr::glr_step_backward_kernel<IO, DECAY, IG><<<static_cast<unsigned>(blocks), glr::kStepThreads, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SSCAN_ERR_CUDA;
    if (!DECAY) return SSCAN_OK;
    const ColumnSums cs = {p.part, {drate, nullptr}, p.B, p.D, 0};
    column_sums_kernel<<<dim3(static_cast<unsigned>(ceil_div(p.D, 32))), kColThreads, 0, s>>>(cs);
    return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

template <class IO>
int forward_t(const glr::FwdParams &p, cudaStream_t s) {
    if (p.rate) return p.igate ? launch_forward<IO, true, true>(p, s) : launch_forward<IO, true, false>(p, s);
    return p.igate ? launch_forward<IO, false, true>(p, s) : launch_forward<IO, false, false>(p, s);
}
template <class IO>
int backward_t(const glr::BwdParams &p, float *drate, cudaStream_t s) {
    if (p.rate)
        return p.igate ? launch_backward<IO, true, true>(p, drate, s) : launch_backward<IO, true, false>(p, drate, s);
    return p.igate ? launch_backward<IO, false, true>(p, drate, s) : launch_backward<IO, false, false>(p, drate, s);
}

}  // namespace

extern "C" {

size_t sscan_glr_states_bytes(int64_t B, int64_t L, int64_t D) {
    if (check_sizes(B, L, D, SSCAN_F32) != SSCAN_OK) return 0;
    return size_t(B) * size_t(runs(L)) * size_t(D) * sizeof(float);
}

int sscan_glr_forward(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate,
                      const void *input_gate, const float *rate, const float *h0, void *y, float *h_final,
                      float *states, void *stream) {
    const int rc = check_sizes(B, L, D, dtype);
    if (rc != SSCAN_OK) return rc;
    const size_t es = dtype == SSCAN_F32 ? 4 : 2;
    const size_t n = size_t(B) * size_t(L) * size_t(D) * es, nh = size_t(B) * size_t(D) * 4;
    if (n && (!x || !gate || !y)) return SSCAN_ERR_INVALID;
    const Span h_out = {h_final == h0 ? nullptr : h_final, nh};  // h_final may be h0's buffer, whole
    const Span ins[] = {{x, n}, {gate, n}, {input_gate, n}, {rate, size_t(D) * 4}, {h0, nh}};
    const Span outs[] = {{y, n}, h_out, {states, sscan_glr_states_bytes(B, L, D)}};
    const int bc = check_buffers(ins, outs, Span{nullptr, 0});
    if (bc != SSCAN_OK) return bc;
    if (h_final && h_final == h0) {  // in place: the other buffers must still be clear of it
        const Span hs = {h_final, nh};
        for (int i = 0; i < 4; ++i)
            if (spans_overlap(hs, ins[i])) return SSCAN_ERR_INVALID;
        if (spans_overlap(hs, outs[0]) || spans_overlap(hs, outs[2])) return SSCAN_ERR_INVALID;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (L == 0) {  // no tokens: the final state is the initial one
        if (!h_final || h_final == h0) return SSCAN_OK;
        const cudaError_t e = h0 ? cudaMemcpyAsync(h_final, h0, nh, cudaMemcpyDeviceToDevice, s)
                                 : cudaMemsetAsync(h_final, 0, nh, s);
        return e == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
    }
    const glr::FwdParams p = {x, gate, input_gate, rate, h0, y, h_final, states, B, L, D, runs(L)};
    return dtype == SSCAN_F32 ? forward_t<float>(p, s) : forward_t<uint16_t>(p, s);
}

size_t sscan_glr_backward_workspace_bytes(int64_t B, int64_t L, int64_t D) {
    if (check_sizes(B, L, D, SSCAN_F32) != SSCAN_OK || L == 0) return 0;
    return round_up_256(size_t(B) * size_t(D) * sizeof(float));
}

int sscan_glr_backward(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate,
                       const void *input_gate, const float *rate, const float *states, const void *dy,
                       const float *dh_final, void *dx, void *dgate, void *dinput_gate, float *drate, float *dh0,
                       void *workspace, void *stream) {
    const int rc = check_sizes(B, L, D, dtype);
    if (rc != SSCAN_OK) return rc;
    const size_t es = dtype == SSCAN_F32 ? 4 : 2;
    const size_t n = size_t(B) * size_t(L) * size_t(D) * es, nh = size_t(B) * size_t(D) * 4;
    if (n && (!x || !gate || !states || !dy || !dx || !dgate)) return SSCAN_ERR_INVALID;
    if (n && (!input_gate != !dinput_gate)) return SSCAN_ERR_INVALID;
    if (!rate != !drate) return SSCAN_ERR_INVALID;
    const size_t wsb = rate ? sscan_glr_backward_workspace_bytes(B, L, D) : 0;
    if (wsb && !workspace) return SSCAN_ERR_WORKSPACE;
    const Span ins[] = {{x, n}, {gate, n}, {input_gate, n}, {rate, size_t(D) * 4},
                        {states, sscan_glr_states_bytes(B, L, D)}, {dy, n}, {dh_final, nh}};
    const Span outs[] = {{dx, n}, {dgate, n}, {dinput_gate, n}, {drate, size_t(D) * 4}, {dh0, nh}};
    const int bc = check_buffers(ins, outs, Span{workspace, wsb});
    if (bc != SSCAN_OK) return bc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (L == 0) {  // no tokens: dh0 = dh_final, and the rate has no part in anything
        if (drate && cudaMemsetAsync(drate, 0, size_t(D) * 4, s) != cudaSuccess) return SSCAN_ERR_CUDA;
        if (dh0 && (dh_final ? cudaMemcpyAsync(dh0, dh_final, nh, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(dh0, 0, nh, s)) != cudaSuccess)
            return SSCAN_ERR_CUDA;
        return SSCAN_OK;
    }
    const glr::BwdParams p = {x, gate, input_gate, dy, rate, states, dh_final, dx, dgate, dinput_gate, dh0,
                              static_cast<float *>(workspace), B, L, D, runs(L)};
    return dtype == SSCAN_F32 ? backward_t<float>(p, drate, s) : backward_t<uint16_t>(p, drate, s);
}

}  // extern "C"
