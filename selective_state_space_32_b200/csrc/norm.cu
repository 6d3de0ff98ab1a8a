// norm.cu -- C ABI of the layer norm (kernels in kernel_norm.cuh): argument checks and
// the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "abi_checks.cuh"
#include "column_sums.cuh"
#include "kernel_norm.cuh"
#include "sscan.h"

using namespace sscan;

namespace {

constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
constexpr int64_t kBwdBlocks = 296;  // backward blocks, each with one row of partial sums per gradient

int check_sizes(int64_t rows, int64_t D, int dtype, uint32_t flags) {
    if (rows < 0 || D < 1) return SSCAN_ERR_INVALID;
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    if (flags & ~static_cast<uint32_t>(SSCAN_NORM_RMS | SSCAN_NORM_RESIDUAL_F32)) return SSCAN_ERR_INVALID;
    if (rows > (int64_t(1) << 40) || D > (int64_t(1) << 31) || (rows > 0 && D > (int64_t(1) << 48) / rows))
        return SSCAN_ERR_UNSUPPORTED;
    return SSCAN_OK;
}

int64_t bwd_blocks(int64_t rows) { return rows < kBwdBlocks ? rows : kBwdBlocks; }

template <class IO, class R, bool RES>
int launch_forward(const norm::FwdParams &p, bool rms, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.rows < kMaxGrid ? p.rows : kMaxGrid);
    if (rms)
        norm::norm_forward_kernel<IO, R, RES, true><<<grid, norm::kRowThreads, 0, s>>>(p);
    else
        norm::norm_forward_kernel<IO, R, RES, false><<<grid, norm::kRowThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

template <class IO, class R>
int launch_backward(const norm::BwdParams &p, bool rms, float *dweight, float *dbias, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(bwd_blocks(p.rows));
    if (rms)
        norm::norm_backward_kernel<IO, R, true><<<grid, norm::kRowThreads, 0, s>>>(p);
    else
        norm::norm_backward_kernel<IO, R, false><<<grid, norm::kRowThreads, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SSCAN_ERR_CUDA;
    if (!dweight && !dbias) return SSCAN_OK;
    const ColumnSums cs = {p.part, {dweight, dbias}, grid, p.D, int64_t(grid) * p.D};
    column_sums_kernel<<<dim3(static_cast<unsigned>(ceil_div(p.D, 32)), 2), kColThreads, 0, s>>>(cs);
    return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

}  // namespace

extern "C" {

int sscan_norm_forward(int64_t rows, int64_t D, int dtype, uint32_t flags, float eps, const void *x,
                       const void *residual, const float *weight, const float *bias, void *y, void *residual_out,
                       float *mean, float *rstd, void *stream) {
    const int rc = check_sizes(rows, D, dtype, flags);
    if (rc != SSCAN_OK) return rc;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return SSCAN_ERR_INVALID;
    const bool rms = flags & SSCAN_NORM_RMS;
    const bool rf32 = dtype == SSCAN_F32 || (flags & SSCAN_NORM_RESIDUAL_F32);
    const size_t n = size_t(rows) * size_t(D), es = dtype == SSCAN_F32 ? 4 : 2, rs = rf32 ? 4 : 2;
    if (n && (!x || !y)) return SSCAN_ERR_INVALID;
    if (n && (!residual != !residual_out)) return SSCAN_ERR_INVALID;
    if (rms && mean) return SSCAN_ERR_INVALID;
    const Span ins[] = {{x, n * es}, {residual, n * rs}, {weight, size_t(D) * 4}, {bias, size_t(D) * 4}};
    const Span outs[] = {{y, n * es}, {residual_out, n * rs}, {mean, size_t(rows) * 4}, {rstd, size_t(rows) * 4}};
    const int bc = check_buffers(ins, outs, Span{nullptr, 0});
    if (bc != SSCAN_OK) return bc;
    if (rows == 0) return SSCAN_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const norm::FwdParams p = {x, residual, weight, bias, y, residual_out, mean, rstd, rows, D, eps};
    if (dtype == SSCAN_F32)
        return residual ? launch_forward<float, float, true>(p, rms, s) : launch_forward<float, float, false>(p, rms, s);
    if (!residual) return launch_forward<uint16_t, uint16_t, false>(p, rms, s);
    return rf32 ? launch_forward<uint16_t, float, true>(p, rms, s) : launch_forward<uint16_t, uint16_t, true>(p, rms, s);
}

size_t sscan_norm_backward_workspace_bytes(int64_t rows, int64_t D) {
    if (check_sizes(rows, D, SSCAN_F32, 0) != SSCAN_OK || rows == 0) return 0;
    return round_up_256(2 * size_t(bwd_blocks(rows)) * size_t(D) * sizeof(float));
}

int sscan_norm_backward(int64_t rows, int64_t D, int dtype, uint32_t flags, const void *dy, const void *s_in,
                        const float *mean, const float *rstd, const float *weight, const void *dresidual, void *ds,
                        void *dx, float *dweight, float *dbias, void *workspace, void *stream) {
    const int rc = check_sizes(rows, D, dtype, flags);
    if (rc != SSCAN_OK) return rc;
    const bool rms = flags & SSCAN_NORM_RMS;
    const bool rf32 = dtype == SSCAN_F32 || (flags & SSCAN_NORM_RESIDUAL_F32);
    const bool two = dtype == SSCAN_BF16 && rf32;  // ds and dx differ in type
    const size_t n = size_t(rows) * size_t(D), es = dtype == SSCAN_F32 ? 4 : 2, rs = rf32 ? 4 : 2;
    if (n && (!dy || !s_in || !rstd || (!rms && !mean) || !ds)) return SSCAN_ERR_INVALID;
    if (rms && mean) return SSCAN_ERR_INVALID;
    if (dx && !two) return SSCAN_ERR_INVALID;
    if (dweight && !weight) return SSCAN_ERR_INVALID;
    const size_t wsb = dweight || dbias ? sscan_norm_backward_workspace_bytes(rows, D) : 0;
    if (wsb && !workspace) return SSCAN_ERR_WORKSPACE;
    const Span ins[] = {{dy, n * es}, {s_in, n * rs}, {mean, size_t(rows) * 4}, {rstd, size_t(rows) * 4},
                        {weight, size_t(D) * 4}, {dresidual, n * rs}};
    const Span outs[] = {{ds, n * rs}, {dx, n * es}, {dweight, size_t(D) * 4}, {dbias, size_t(D) * 4}};
    const int bc = check_buffers(ins, outs, Span{workspace, wsb});
    if (bc != SSCAN_OK) return bc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // no rows: the sums are empty
        if (dweight && cudaMemsetAsync(dweight, 0, size_t(D) * 4, s) != cudaSuccess) return SSCAN_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, size_t(D) * 4, s) != cudaSuccess) return SSCAN_ERR_CUDA;
        return SSCAN_OK;
    }
    const norm::BwdParams p = {dy, s_in, dresidual, mean, rstd, weight, ds, dx, static_cast<float *>(workspace),
                               rows, D, dweight != nullptr, dbias != nullptr};
    if (dtype == SSCAN_F32) return launch_backward<float, float>(p, rms, dweight, dbias, s);
    return rf32 ? launch_backward<uint16_t, float>(p, rms, dweight, dbias, s)
                : launch_backward<uint16_t, uint16_t>(p, rms, dweight, dbias, s);
}

}  // extern "C"
