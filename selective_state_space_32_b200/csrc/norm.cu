// norm.cu -- C ABI of the layer norm (kernels in kernel_norm.cuh): argument checks and
// the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "abi_checks.cuh"
#include "column_sums.cuh"
#include "device_utils.cuh"
#include "kernel_norm.cuh"
#include "sscan.h"

using namespace sscan;

namespace {

int check_sizes(int64_t rows, int64_t D, int dtype, uint32_t flags) {
    if (rows < 0 || D < 1) return SSCAN_ERR_INVALID;
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    if (flags & ~static_cast<uint32_t>(SSCAN_NORM_RMS | SSCAN_NORM_RESIDUAL_F32)) return SSCAN_ERR_INVALID;
    if (rows >= (int64_t(1) << 31) || D > (int64_t(1) << 28)) return SSCAN_ERR_UNSUPPORTED;  // a block a row at most
    return SSCAN_OK;
}

// How a row is shared out: NV vectors of `ve` values a thread, `threads` threads a row (up
// to 32: groups of lanes; more: a block a row), or nv = 0: too long for registers.  Rows of a
// width that is not a multiple of 16 bytes: `shift`, by the aligned vectors that cover them
// (4000 x 6001 bf16 with a residual, forward, 70 us; value by value 147), or value by value
// where one warp takes a row.
struct RowShape {
    int ve, nv, threads;
    bool shift = false;
};
int64_t row_vectors(int64_t D, int ve, bool shift) { return shift ? ceil_div(D + ve - 1, ve) : D / ve; }
RowShape row_shape(int64_t D, int es) {
    const int ve = 16 / es;
    const bool shift = D * es % 16 != 0;
    if (shift && D <= 256) return {1, 8, 32};
    const int64_t n = row_vectors(D, ve, shift);
    if (!shift) {
        if (n <= 8) return {ve, 1, 8};
        if (n <= 16) return {ve, 1, 16};
        if (n <= 32) return {ve, 1, 32};
        if (n <= 64) return {ve, 2, 32};
        if (n <= 128) return {ve, 4, 32};
        if (es == 4 && n <= 256) return {ve, 8, 32};
    }
    if (n <= 256) return {ve, 1, static_cast<int>(ceil_div(n, 32) * 32), shift};
    if (n <= 1024) return {ve, 2, static_cast<int>(ceil_div(n, 64) * 32), shift};
    if (n <= 4 * norm::kMaxThreads) return {ve, 4, static_cast<int>(ceil_div(n, 128) * 32), shift};
    return {shift ? 1 : ve, 0, 0};
}

template <int N> using Int = std::integral_constant<int, N>;

// f(VE, NV, G) with the shape's constants
template <int ES, class F>
int with_shape(const RowShape &sh, F f) {
    constexpr int V = 16 / ES;
    const bool group = sh.threads <= 32;
    if (sh.ve == 1) return f(Int<1>{}, Int<8>{}, Int<32>{});
    if (sh.threads == 8) return f(Int<V>{}, Int<1>{}, Int<8>{});
    if (sh.threads == 16) return f(Int<V>{}, Int<1>{}, Int<16>{});
    if (sh.nv == 1) return group ? f(Int<V>{}, Int<1>{}, Int<32>{}) : f(Int<V>{}, Int<1>{}, Int<0>{});
    if (sh.nv == 2) return group ? f(Int<V>{}, Int<2>{}, Int<32>{}) : f(Int<V>{}, Int<2>{}, Int<0>{});
    if constexpr (ES == 4)
        if (sh.nv == 8) return f(Int<V>{}, Int<8>{}, Int<32>{});
    return group ? f(Int<V>{}, Int<4>{}, Int<32>{}) : f(Int<V>{}, Int<4>{}, Int<0>{});
}

template <class IO, class R, bool RES>
int launch_forward(const norm::FwdParams &p, cudaStream_t s) {
    const RowShape sh = row_shape(p.D, sizeof(IO));
    if (sh.nv == 0) {
        const unsigned blocks = static_cast<unsigned>(p.rows);
        if (sh.ve == 1) norm::norm_forward_long_kernel<IO, R, RES, 1><<<blocks, norm::kLongThreads, 0, s>>>(p);
        else norm::norm_forward_long_kernel<IO, R, RES, 16 / sizeof(IO)><<<blocks, norm::kLongThreads, 0, s>>>(p);
    } else {
        with_shape<sizeof(IO)>(sh, [&](auto ve, auto nv, auto g) {
            constexpr int rows = g ? 128 / (g ? g : 1) : 1;  // of a block
            const unsigned blocks = static_cast<unsigned>(ceil_div(p.rows, rows));
            if constexpr (!g) {
                if (sh.shift) {
                    norm::norm_forward_kernel<IO, R, RES, ve, nv, g, true><<<blocks, sh.threads, 0, s>>>(p);
                    return 0;
                }
            }
            if constexpr (g || nv > 1 || sizeof(IO) == 2)  // aligned fp32 rows of 256 vectors are a warp's
                norm::norm_forward_kernel<IO, R, RES, ve, nv, g, false><<<blocks, rows * sh.threads, 0, s>>>(p);
            return 0;
        });
    }
    return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

// The backward pass holds two sums a value in registers, so a thread takes 16 values at
// most, and its rows go through shared memory.
constexpr int64_t kRingBytes = 220 << 10;
// Shared memory of a block of `rows` rows at a time with rings of `stages` rows
template <class IO, class R>
int64_t bwd_smem(int64_t D, int ve, bool dres, int rows, int stages) {
    const int64_t weight = (D * 4 + 15) / 16 * 16, sums = rows > 1 ? rows * D * 4 : 0;
    const int64_t ring = ve > 1 ? rows * stages * norm::bwd_row_bytes<IO, R>(D, dres) : 0;
    return weight + (ring > sums ? ring : sums);
}
template <class IO, class R>
RowShape bwd_row_shape(int64_t D, bool dres) {
    const RowShape sh = row_shape(D, sizeof(IO));
    if (sh.ve == 1 || sh.nv == 0) return sh;
    const int64_t n = row_vectors(D, sh.ve, sh.shift), smem = bwd_smem<IO, R>(n * sh.ve, sh.ve, dres, 1, norm::kBlockStages);
    const int most = 16 / sh.ve;  // vectors a thread
    if (bwd_smem<IO, R>(n * sh.ve, sh.ve, dres, 1, norm::kLongStages) > kRingBytes || n > int64_t(most) * norm::kBwdThreads)
        return {sh.shift ? 1 : sh.ve, 0, 0};
    if (sh.threads <= 32 && sh.nv <= most) return sh;
    // as few values a thread as leaves the SM's threads to as many rows as its shared memory holds
    const int64_t want = norm::kBwdThreads / (smem * 2 > kRingBytes ? 1 : smem * 4 > kRingBytes ? 2 : 4);
    int nv = 1;
    while (nv < most && n > want * nv) nv *= 2;
    return {sh.ve, nv, static_cast<int>(ceil_div(n, 32 * nv) * 32), sh.shift};
}

// Backward blocks, each leaving one row of partial sums per gradient; where a row takes several
// passes, so many that the rows a block reads twice stay in the L2.
constexpr int64_t kMaxBwdBlocks = 148 * 4, kLongBwdBlocks = 148;
int64_t most_bwd_blocks(int64_t D) {  // of any types
    for (bool dres : {false, true})
        if (bwd_row_shape<float, float>(D, dres).nv || bwd_row_shape<uint16_t, uint16_t>(D, dres).nv ||
            bwd_row_shape<uint16_t, float>(D, dres).nv)
            return kMaxBwdBlocks;
    return kLongBwdBlocks;
}
constexpr int kBwdGroupThreads = 256;  // of a block of several rows

template <class IO, class R>
int launch_backward(const norm::BwdParams &p, float *dweight, float *dbias, cudaStream_t s) {
    const RowShape sh = bwd_row_shape<IO, R>(p.D, p.dresidual != nullptr);
    const int block_rows = sh.nv != 0 && sh.threads <= 32 ? kBwdGroupThreads / sh.threads : 1;
    int64_t blocks = ceil_div(p.rows, block_rows);
    int rc = SSCAN_OK;
    auto at_most = [&](int64_t n) { blocks = blocks < n ? blocks : n; };
    if (sh.nv == 0) {
        at_most(kLongBwdBlocks);
        const int64_t each = ceil_div(p.rows, blocks);
        blocks = ceil_div(p.rows, each);
        const unsigned n = static_cast<unsigned>(blocks);
        if (sh.ve == 1) norm::norm_backward_long_kernel<IO, R, 1><<<n, norm::kLongThreads, 0, s>>>(p, each);
        else norm::norm_backward_long_kernel<IO, R, 16 / sizeof(IO)><<<n, norm::kLongThreads, 0, s>>>(p, each);
    } else {
        rc = with_shape<sizeof(IO)>(sh, [&](auto ve, auto nv, auto g) -> int {
            if constexpr (ve * nv > 16) {
                return SSCAN_ERR_INVALID;  // not a shape of bwd_row_shape
            } else {
                const bool dres = p.dresidual != nullptr;
                const int threads = g ? kBwdGroupThreads : sh.threads;
                const int64_t width = ve > 1 ? row_vectors(p.D, ve, sh.shift) * ve : p.D;
                auto launch_as = [&](auto stages, auto shift) -> int {
                    constexpr auto kern = norm::norm_backward_kernel<IO, R, ve, nv, g, stages, shift>;
                    const int64_t smem = bwd_smem<IO, R>(width, ve, dres, block_rows, stages);
                    int per_sm = static_cast<int>((kRingBytes + 7 * 1024) / (smem + 1024));  // blocks of an SM
                    if (per_sm * threads > norm::kBwdThreads) per_sm = norm::kBwdThreads / threads;
                    at_most(148 * (per_sm < 1 ? 1 : per_sm > 4 ? 4 : per_sm));
                    if (shift && blocks < p.rows) blocks -= blocks % ve;  // a block's rows begin alike
                    if (smem_opt_in<kern>(static_cast<int>(kRingBytes)) != cudaSuccess) return SSCAN_ERR_CUDA;
                    kern<<<static_cast<unsigned>(blocks), threads, smem, s>>>(p);
                    return SSCAN_OK;
                };
                auto launch = [&](auto stages) -> int {
                    if constexpr (!g)
                        if (sh.shift) return launch_as(stages, Int<1>{});
                    return launch_as(stages, Int<0>{});
                };
                // rows that fill shared memory take 16 values a thread, and some types' never do
                constexpr int64_t widest = 16 * norm::kBwdThreads;
                constexpr bool fills = ve > 1 && ve * nv == 16 &&
                                       widest * 4 + norm::kBlockStages * norm::bwd_row_bytes<IO, R>(widest, true) > kRingBytes;
                if constexpr (g) {
                    return launch(Int<norm::kGroupStages>{});
                } else {
                    if constexpr (fills)
                        if (bwd_smem<IO, R>(width, ve, dres, 1, norm::kBlockStages) > kRingBytes)
                            return launch(Int<norm::kLongStages>{});
                    return launch(Int<norm::kBlockStages>{});
                }
            }
        });
    }
    if (rc != SSCAN_OK) return rc;
    if (cudaGetLastError() != cudaSuccess) return SSCAN_ERR_CUDA;
    if (!dweight && !dbias) return SSCAN_OK;
    const ColumnSums cs = {p.part, {dweight, dbias}, blocks, p.D, blocks * p.D};
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
    const norm::FwdParams p = {x, residual, weight, bias, y, residual_out, mean, rstd, rows, D, eps, rms};
    if (dtype == SSCAN_F32)
        return residual ? launch_forward<float, float, true>(p, s) : launch_forward<float, float, false>(p, s);
    if (!residual) return launch_forward<uint16_t, uint16_t, false>(p, s);
    return rf32 ? launch_forward<uint16_t, float, true>(p, s) : launch_forward<uint16_t, uint16_t, true>(p, s);
}

size_t sscan_norm_backward_workspace_bytes(int64_t rows, int64_t D) {
    if (check_sizes(rows, D, SSCAN_F32, 0) != SSCAN_OK || rows == 0) return 0;
    const int64_t most = most_bwd_blocks(D);
    return round_up_256(2 * size_t(rows < most ? rows : most) * size_t(D) * sizeof(float));
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
                               rows, D, rms, dweight != nullptr, dbias != nullptr};
    if (dtype == SSCAN_F32) return launch_backward<float, float>(p, dweight, dbias, s);
    return rf32 ? launch_backward<uint16_t, float>(p, dweight, dbias, s)
                : launch_backward<uint16_t, uint16_t>(p, dweight, dbias, s);
}

}  // extern "C"
