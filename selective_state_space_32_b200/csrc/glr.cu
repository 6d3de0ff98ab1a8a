// glr.cu -- C ABI of the gated linear recurrence (kernels in kernel_glr.cuh): argument
// checks, the choice of the kernel and the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "abi_checks.cuh"
#include "column_sums.cuh"
#include "kernel_glr.cuh"
#include "kernel_glr_scan.cuh"
#include "sscan.h"

using namespace sscan;

namespace {

// Sizes that every index and grid of the kernels can hold.
int check_sizes(int64_t B, int64_t L, int64_t D, int dtype) {
    if (B < 1 || D < 1 || L < 0) return SSCAN_ERR_INVALID;
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    const int64_t kMax = int64_t(1) << 31;
    if (B >= kMax || D > (int64_t(1) << 28) || B * D >= kMax) return SSCAN_ERR_UNSUPPORTED;
    if (L > (int64_t(1) << 40) || (L > 0 && B * D > (int64_t(1) << 48) / L)) return SSCAN_ERR_UNSUPPORTED;
    return SSCAN_OK;
}

// Up to this many tokens the forward pass takes one thread per channel pair: 128 rows of 8
// tokens, 2048 channels 5.8 us against 10.9 of the scan; 16 tokens of 8 rows 4.8 against 2.9.
constexpr int64_t kStepTokens = 8;

int64_t runs(int64_t L) { return ceil_div(L, glr::kRun); }

// How a walk is spread along the sequence: warps of a block, blocks of a cluster.
struct Shape {
    int warps, cluster;
};

// `chains` = batch rows times channel groups, `n` = runs of the sequence.  Measured on B200
// (us; warps x blocks): about ten warps an SM are wanted, in small blocks first: 192 chains of
// 2048 tokens, bf16 with rate and input gate: 4x2 51, 4x1 64, 8x4 58; 384 fp32 chains: 4x1 49,
// 8x1 56, 4x2 62; 128 chains of 8192 tokens: 4x4 73, 4x2 87, 8x8 94.  With enough chains,
// blocks of 8 warps instead of clusters of two (384 fp32 chains, backward: 8x1 84, 4x2 86).
// Where clusters of 8 small blocks leave the device half empty, 8 warps as well (32 chains of
// 131072 tokens, backward: 8x8 1154, 4x8 1375; forward the other way, 631 and 597), and for a
// handful of chains clusters of 16 (1 chain of 65536 tokens: 8x16 95, 8x8 205).  With very
// many chains fewer warps share one.
struct Fill {
    int64_t want, low;  // warps that fill the device, and too few of them in blocks of 4
};
Shape scan_shape(int64_t chains, int64_t n, const Fill &fill) {
    int w = 1;
    while (w < 4 && w < n) w *= 2;
    while (w > 1 && chains * w >= 16384) w /= 2;
    auto cluster = [&](int most) {
        int c = 1;
        while (c < most && c * w < n && chains * w * c < fill.want) c *= 2;
        return c;
    };
    int c = cluster(8);
    if (w == 4 && c == 2 && chains >= 2 * 148) w = glr::kMaxWarps, c = 1;
    if (w * c < n && chains * w * c < fill.low) w = glr::kMaxWarps, c = cluster(8);
    if (w * c < n && chains * w * c < fill.want / 4) c = cluster(glr::kMaxCluster);
    return {w, c};
}
// Without staged loads a warp waits for its inputs in every step, and more warps pay: 196
// chains of 2000 tokens of odd width, bf16 with both gates: 4x4 52 us, 4x2 85.
constexpr Fill forward_fill(bool staged) { return {148 * (staged ? 10 : 11), 148 * 6}; }
constexpr Fill backward_fill(bool staged, int blocks) {
    const int64_t want = 148 * (!staged ? 11 : blocks == 3 ? 13 : 10);
    return {want, want};
}

template <class IO>
bool staged(int64_t D) { return D * int64_t(sizeof(IO)) % 16 == 0; }

// Dynamic shared memory, and clusters of more than 8 blocks, for kernel KERN: once per
// (kernel, device) as smem_opt_in does.
template <auto KERN>
cudaError_t cluster_opt_in(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(KERN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// Blocks, cluster and shared memory of a scan kernel's launch, on stream s.
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    Launch(int64_t blocks, const Shape &sh, int smem, cudaStream_t s) {
        cfg.gridDim = dim3(static_cast<unsigned>(blocks));
        cfg.blockDim = dim3(32 * sh.warps);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = sh.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = sh.cluster > 1 ? 1 : 0;
    }
};

template <class IO, int V, bool STAGED, bool DECAY, bool IG>
int launch_scan(const glr::FwdParams &p, const glr::Waits &waits, cudaStream_t s) {
    constexpr int NS = IG ? 3 : 2, K = glr::kForwardRun;
    const int64_t groups = ceil_div(p.D, 32 * V);
    const Shape sh = scan_shape(p.B * groups, ceil_div(p.L, K), forward_fill(STAGED));
    constexpr auto kern = glr::glr_scan_kernel<IO, V, STAGED, DECAY, IG, K>;
    if (cluster_opt_in<kern>(glr::scan_smem_bytes<IO, V, STAGED, NS, K>(glr::kMaxWarps, glr::kMaxCluster)) != cudaSuccess)
        return SSCAN_ERR_CUDA;
    Launch l(p.B * groups * sh.cluster, sh, glr::scan_smem_bytes<IO, V, STAGED, NS, K>(sh.warps, sh.cluster), s);
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, p, waits, groups, static_cast<uint32_t>(sh.cluster));
    return e == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

template <class IO, bool DECAY, bool IG>
int launch_forward(const glr::FwdParams &p, const glr::Waits &waits, cudaStream_t s) {
    if (p.L <= kStepTokens) {
        const bool pairs = p.D % 2 == 0;
        const unsigned blocks = static_cast<unsigned>(ceil_div(p.B * p.D, (pairs ? 2 : 1) * glr::kStepThreads));
        if (pairs)
            glr::glr_step_kernel<IO, 2, DECAY, IG><<<blocks, glr::kStepThreads, 0, s>>>(p);
        else
            glr::glr_step_kernel<IO, 1, DECAY, IG><<<blocks, glr::kStepThreads, 0, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
    }
    if (!staged<IO>(p.D)) return launch_scan<IO, 1, false, DECAY, IG>(p, waits, s);
    return launch_scan<IO, glr::lane_channels<IO, true>(), true, DECAY, IG>(p, waits, s);
}

template <class IO, int V, bool STAGED, bool DECAY, bool IG>
int launch_scan_backward(const glr::BwdParams &p, const glr::Waits &waits, float *drate, cudaStream_t s) {
    constexpr int NS = IG ? 4 : 3, K = glr::kRun;
    const int64_t groups = ceil_div(p.D, 32 * V);
    const Shape sh = scan_shape(p.B * groups, p.nruns, backward_fill(STAGED, glr::scan_blocks<V>()));
    constexpr auto kern = glr::glr_scan_backward_kernel<IO, V, STAGED, DECAY, IG>;
    if (cluster_opt_in<kern>(glr::scan_smem_bytes<IO, V, STAGED, NS, K>(glr::kMaxWarps, glr::kMaxCluster)) != cudaSuccess)
        return SSCAN_ERR_CUDA;
    Launch l(p.B * groups * sh.cluster, sh, glr::scan_smem_bytes<IO, V, STAGED, NS, K>(sh.warps, sh.cluster), s);
    if (cudaLaunchKernelEx(&l.cfg, kern, p, waits, groups, static_cast<uint32_t>(sh.cluster)) != cudaSuccess)
        return SSCAN_ERR_CUDA;
    if (!DECAY) return SSCAN_OK;
    const ColumnSums cs = {p.part, {drate, nullptr}, p.B * sh.cluster, p.D, 0};
    column_sums_kernel<<<dim3(static_cast<unsigned>(ceil_div(p.D, 32))), kColThreads, 0, s>>>(cs);
    return cudaGetLastError() == cudaSuccess ? SSCAN_OK : SSCAN_ERR_CUDA;
}

template <class IO, bool DECAY, bool IG>
int launch_backward(const glr::BwdParams &p, const glr::Waits &waits, float *drate, cudaStream_t s) {
    if (!staged<IO>(p.D)) return launch_scan_backward<IO, 1, false, DECAY, IG>(p, waits, drate, s);
    return launch_scan_backward<IO, glr::lane_channels<IO, true>(), true, DECAY, IG>(p, waits, drate, s);
}

template <class IO>
int forward_t(const glr::FwdParams &p, const glr::Waits &waits, cudaStream_t s) {
    if (p.rate)
        return p.igate ? launch_forward<IO, true, true>(p, waits, s) : launch_forward<IO, true, false>(p, waits, s);
    return p.igate ? launch_forward<IO, false, true>(p, waits, s) : launch_forward<IO, false, false>(p, waits, s);
}
template <class IO>
int backward_t(const glr::BwdParams &p, const glr::Waits &waits, float *drate, cudaStream_t s) {
    if (p.rate)
        return p.igate ? launch_backward<IO, true, true>(p, waits, drate, s)
                       : launch_backward<IO, true, false>(p, waits, drate, s);
    return p.igate ? launch_backward<IO, false, true>(p, waits, drate, s)
                   : launch_backward<IO, false, false>(p, waits, drate, s);
}

size_t states_bytes(int64_t B, int64_t L, int64_t D) {
    if (check_sizes(B, L, D, SSCAN_F32) != SSCAN_OK) return 0;
    return size_t(B) * size_t(runs(L)) * size_t(D) * sizeof(float);
}

// A status word is 4-byte aligned and clear of every other buffer.
template <int NI, int NO>
int check_status(const int *status, const Span (&ins)[NI], const Span (&outs)[NO], const Span &ws) {
    if (reinterpret_cast<uintptr_t>(status) & 3u) return SSCAN_ERR_ALIGN;
    const Span st = {status, sizeof(int)};
    for (const Span &s : ins)
        if (spans_overlap(st, s)) return SSCAN_ERR_INVALID;
    for (const Span &s : outs)
        if (spans_overlap(st, s)) return SSCAN_ERR_INVALID;
    return spans_overlap(st, ws) ? SSCAN_ERR_WORKSPACE : SSCAN_OK;
}

int forward(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate, const void *input_gate,
            const float *rate, const float *h0, void *y, float *h_final, float *states, const glr::Waits &waits,
            void *stream) {
    const int rc = check_sizes(B, L, D, dtype);
    if (rc != SSCAN_OK) return rc;
    const size_t es = dtype == SSCAN_F32 ? 4 : 2;
    const size_t n = size_t(B) * size_t(L) * size_t(D) * es, nh = size_t(B) * size_t(D) * 4;
    if (n && (!x || !gate || !y)) return SSCAN_ERR_INVALID;
    const Span h_out = {h_final == h0 ? nullptr : h_final, nh};  // h_final may be h0's buffer, whole
    const Span ins[] = {{x, n}, {gate, n}, {input_gate, n}, {rate, size_t(D) * 4}, {h0, nh}};
    const Span outs[] = {{y, n}, h_out, {states, states_bytes(B, L, D)}};
    int bc = check_buffers(ins, outs, Span{nullptr, 0});
    if (bc == SSCAN_OK) bc = check_status(waits.status, ins, outs, Span{nullptr, 0});
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
    return dtype == SSCAN_F32 ? forward_t<float>(p, waits, s) : forward_t<uint16_t>(p, waits, s);
}

size_t workspace_bytes(int64_t B, int64_t L, int64_t D) {
    if (check_sizes(B, L, D, SSCAN_F32) != SSCAN_OK || L == 0) return 0;
    // one row of D sums per block of a walk, for whichever of the types and widths' kernels runs
    const int64_t n = runs(L), narrow = B * ceil_div(D, 32), wide = B * ceil_div(D, 64);
    int c = scan_shape(wide, n, backward_fill(true, glr::scan_blocks<2>())).cluster;
    for (bool st : {false, true}) {
        const int k = scan_shape(narrow, n, backward_fill(st, glr::scan_blocks<1>())).cluster;
        c = k > c ? k : c;
    }
    return round_up_256(size_t(B) * size_t(c) * size_t(D) * sizeof(float));
}

int backward(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate, const void *input_gate,
             const float *rate, const float *states, const void *dy, const float *dh_final, void *dx, void *dgate,
             void *dinput_gate, float *drate, float *dh0, void *workspace, const glr::Waits &waits, void *stream) {
    const int rc = check_sizes(B, L, D, dtype);
    if (rc != SSCAN_OK) return rc;
    const size_t es = dtype == SSCAN_F32 ? 4 : 2;
    const size_t n = size_t(B) * size_t(L) * size_t(D) * es, nh = size_t(B) * size_t(D) * 4;
    if (n && (!x || !gate || !states || !dy || !dx || !dgate)) return SSCAN_ERR_INVALID;
    if (n && (!input_gate != !dinput_gate)) return SSCAN_ERR_INVALID;
    if (!rate != !drate) return SSCAN_ERR_INVALID;
    const size_t wsb = rate ? workspace_bytes(B, L, D) : 0;
    if (wsb && !workspace) return SSCAN_ERR_WORKSPACE;
    const Span ins[] = {{x, n}, {gate, n}, {input_gate, n}, {rate, size_t(D) * 4},
                        {states, states_bytes(B, L, D)}, {dy, n}, {dh_final, nh}};
    const Span outs[] = {{dx, n}, {dgate, n}, {dinput_gate, n}, {drate, size_t(D) * 4}, {dh0, nh}};
    int bc = check_buffers(ins, outs, Span{workspace, wsb});
    if (bc == SSCAN_OK) bc = check_status(waits.status, ins, outs, Span{workspace, wsb});
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
    return dtype == SSCAN_F32 ? backward_t<float>(p, waits, drate, s) : backward_t<uint16_t>(p, waits, drate, s);
}

}  // namespace

extern "C" {

size_t sscan_glr_states_bytes(int64_t B, int64_t L, int64_t D) { return states_bytes(B, L, D); }

int sscan_glr_forward(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate,
                      const void *input_gate, const float *rate, const float *h0, void *y, float *h_final,
                      float *states, void *stream) {
    return forward(B, L, D, dtype, x, gate, input_gate, rate, h0, y, h_final, states, {nullptr, kSpinLimit}, stream);
}

int sscan_glr_forward_checked(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate,
                              const void *input_gate, const float *rate, const float *h0, void *y, float *h_final,
                              float *states, int *status, uint32_t tries, void *stream) {
    return forward(B, L, D, dtype, x, gate, input_gate, rate, h0, y, h_final, states,
                   {status, tries < kSpinLimit ? tries : kSpinLimit}, stream);
}

size_t sscan_glr_backward_workspace_bytes(int64_t B, int64_t L, int64_t D) { return workspace_bytes(B, L, D); }

int sscan_glr_backward(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate,
                       const void *input_gate, const float *rate, const float *states, const void *dy,
                       const float *dh_final, void *dx, void *dgate, void *dinput_gate, float *drate, float *dh0,
                       void *workspace, void *stream) {
    return backward(B, L, D, dtype, x, gate, input_gate, rate, states, dy, dh_final, dx, dgate, dinput_gate, drate, dh0,
                    workspace, {nullptr, kSpinLimit}, stream);
}

int sscan_glr_backward_checked(int64_t B, int64_t L, int64_t D, int dtype, const void *x, const void *gate,
                               const void *input_gate, const float *rate, const float *states, const void *dy,
                               const float *dh_final, void *dx, void *dgate, void *dinput_gate, float *drate,
                               float *dh0, void *workspace, int *status, uint32_t tries, void *stream) {
    return backward(B, L, D, dtype, x, gate, input_gate, rate, states, dy, dh_final, dx, dgate, dinput_gate, drate, dh0,
                    workspace, {status, tries < kSpinLimit ? tries : kSpinLimit}, stream);
}

}  // extern "C"
