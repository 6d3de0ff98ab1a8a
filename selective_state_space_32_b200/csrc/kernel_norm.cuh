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
// backward pass reads.  They come from centred squares, so that a mean far from zero costs
// no digits of the variance.
//
// Both passes are streams: a row is read once, held in registers, and written once.  T
// threads share a row, in vectors of VE consecutive values (16 bytes of x; single values in
// short rows whose D is not a multiple), NV vectors a thread: thread i takes vectors i, i + T,
// ...  A short row belongs to a group of G = 8, 16 or 32 lanes (no barrier at all); a longer
// one is the block's (G = 0), which meets once: each warp reduces its own part (forward: mean and centred squares,
// joined by (n, mean, M2) as of sets; backward: two sums), and every thread joins the
// warps' results in the same order.
//
// The backward pass's blocks stay and walk the rows, so that a thread keeps its columns'
// dw and db in registers; a block leaves one row of partial sums, and the next rows'
// inputs are in flight while a row is worked on.
//
// What bounds it (B200; share of the copy rate).  Forward: HBM (32768 x 2048 bf16 with an fp32
// residual 118 us, 106 %; 16384 x 5120 bf16 101 us, 103 %; 16384 x 768 fp32 18 us, 87 %;
// 65536 x 256 bf16 25 us, 83 %).  Backward, with the columns' sums: HBM for long rows with an
// fp32 stream (32768 x 2048 165 us, 101 %; 8192 x 4096 fp32 85 us, 98 %), the two reductions
// and the shared-memory reads of a row otherwise (16384 x 5120 bf16 134 us, 77 %; 32768 x 1024
// bf16 56 us, 74 %; 16384 x 768 bf16 39 us, 79 %).  Widths that are not a multiple of 16 bytes, by
// the aligned vectors that cover a row: 4000 x 6001 bf16 with a residual 70 and 81 us (42 and
// 37 %), 4000 x 7999 with an fp32 one 96 and 176, 8000 x 1999 41 and 49, 2001 x 777 fp32 8 and 12;
// value by value 147 and 223, 166 and 322, 60 and 74, 7.5 and 12.5.  What holds them: forward 51 to
// 63 registers against 32, so half the warps; backward with 16 values a thread 72 to 276 bytes of
// registers spilled under the 96 that 640 threads leave.
//
// The rings are addressed by 32-bit shared addresses; as pointers, their 64-bit arithmetic was
// 5 of 35 instructions a value (16384 x 5120 142 us, 16384 x 768 50 us).
#pragma once

#include "cp_async.cuh"
#include "device_utils.cuh"

namespace sscan {
namespace norm {

struct FwdParams {
    const void *x, *residual;
    const float *weight, *bias;
    void *y, *residual_out;
    float *mean, *rstd;
    int64_t rows, D;
    float eps;
    int rms;
};

struct BwdParams {
    const void *dy, *s, *dresidual;
    const float *mean, *rstd, *weight;
    void *ds, *dx;  // ds in s's type; dx in dy's type (null: the same type, ds serves)
    float *part;    // [2][gridDim.x][D]: dw, db of each block's rows
    int64_t rows, D;
    int rms, want_dw, want_db;
};

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float inv_sqrt(float v) { return 1.0f / sqrtf(v); }
// Sum over groups of G lanes, the same value in each lane of a group
template <int G = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// VE consecutive values of type T as loaded, and as fp32
template <class T, int VE> struct Raw {
    static constexpr int kWords = VE * Io<T>::kBytes / 4;  // 0 with VE = 1 of bf16
    uint32_t w[kWords > 0 ? kWords : 1];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VE == 1) {
            if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(Io<T>::ld(p));
            else w[0] = Io<T>::ld(p);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        }
    }
    // from shared memory, at a 32-bit shared address
    __device__ __forceinline__ void load_shared(uint32_t p) {
        if constexpr (VE == 1) {
            if constexpr (sizeof(T) == 4) {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p) : "memory");
            } else {
                asm volatile("{\n\t.reg .b16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(w[0]) : "r"(p) : "memory");
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                             : "r"(p + 16 * i)
                             : "memory");
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (uint32_t &x : w) x = 0;
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        else return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[VE]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < VE; ++e) w[e] = __float_as_uint(v[e]);
        } else if constexpr (VE == 1) {
            asm("{\n\t.reg .b16 h;\n\tcvt.rn.bf16.f32 h, %1;\n\tmov.b32 %0, {h, 0};\n\t}" : "=r"(w[0]) : "f"(v[0]));
        } else {
#pragma unroll
            for (int e = 0; e < VE; e += 2)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e / 2]) : "f"(v[e + 1]), "f"(v[e]));
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VE == 1) {
            if constexpr (sizeof(T) == 4) *p = __uint_as_float(w[0]);
            else *p = static_cast<uint16_t>(w[0]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
};

// Rows that do not begin at a 16-byte boundary (SHIFT): a row of D values from value `row0` on is
// covered by the aligned vectors from row0 - m on, m = row0 % VE; value e of vector j is column
// j VE - m + e, and the first and the last vector hold values of other rows too.  A vector that
// reaches past the tensor's `total` values is read value by value.
template <class T, int VE>
__device__ __forceinline__ void load_shifted(Raw<T, VE> &q, const T *p, int64_t at, int64_t total) {
    if (at + VE <= total) {
        q.load(p + at);
        return;
    }
    float v[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) v[e] = at + e < total ? Io<T>::widen(Io<T>::ld(p + at + e)) : 0.0f;
    q.set(v);
}
// VE weights from column c on (0 for columns that are none): aligned vectors of four, and the
// values picked from them; c % 4 is the same in a block.
template <int VE>
__device__ __forceinline__ void weights_shifted(float (&o)[VE], const float *p, int64_t c, int64_t D) {
    const int sh = static_cast<int>(c & 3);
    if (c < 0 || c - sh + VE + 4 > D) {
#pragma unroll
        for (int e = 0; e < VE; ++e) o[e] = c + e >= 0 && c + e < D ? __ldg(p + c + e) : 0.0f;
        return;
    }
    Raw<float, VE + 4> q;
    q.load(p + c - sh);
    float v[VE + 2];
#pragma unroll
    for (int e = 0; e < VE + 2; ++e) v[e] = sh & 1 ? q.get(e + 1) : q.get(e);
#pragma unroll
    for (int e = 0; e < VE; ++e) o[e] = sh & 2 ? v[e + 2] : v[e];
}

// values of a row that warp w of a row of T threads holds
template <int VE, int NV>
__device__ __forceinline__ int warp_values(int64_t nvec, int w, int T) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t left = nvec - (w * 32 + static_cast<int64_t>(i) * T);
        n += left >= 32 ? 32 : left > 0 ? static_cast<int>(left) : 0;
    }
    return n * VE;
}

// IO: x, y; R: residual and residual_out.  G > 0: blockDim / G rows a block; G = 0: one.
template <class IO, class R, bool RES, int VE, int NV, int G, bool SHIFT>
__global__ void __launch_bounds__(G ? 128 : kMaxThreads) norm_forward_kernel(const FwdParams p) {
    static_assert(!SHIFT || (G == 0 && VE > 1), "a block a row, by vectors");
    __shared__ float4 part[32];  // a warp's number of values, their mean and centred squares
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int T = G ? G : blockDim.x, t = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
    const int64_t row = G ? (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / (G ? G : 1) : blockIdx.x;
    // groups past the last row go along with nothing to read or write
    const int m = SHIFT ? static_cast<int>(row * p.D % VE) : 0;
    const int64_t nvec = SHIFT ? (p.D + m + VE - 1) / VE : row < p.rows ? p.D / VE : 0, at = row * p.D - m;
    const int64_t total = p.rows * p.D;
    // the first vector of others' values at its start, the last of others' at its end
    auto edge = [&](int64_t j) { return SHIFT && (j == 0 || j == nvec - 1); };
    auto inside = [&](int64_t j, int e) { return j * VE + e >= m && j * VE + e < p.D + m; };
    float v[NV][VE];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t j = t + static_cast<int64_t>(i) * T;
        Raw<IO, VE> x;
        x.zero();
        if (j < nvec) {
            if constexpr (SHIFT) load_shifted(x, static_cast<const IO *>(p.x), at + j * VE, total);
            else x.load(static_cast<const IO *>(p.x) + at + j * VE);
        }
        if constexpr (RES) {
            Raw<R, VE> r;
            r.zero();
            if (j < nvec) {
                if constexpr (SHIFT) load_shifted(r, static_cast<const R *>(p.residual), at + j * VE, total);
                else r.load(static_cast<const R *>(p.residual) + at + j * VE);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = x.get(e) + r.get(e);
            r.set(v[i]);
            R *out = static_cast<R *>(p.residual_out) + at + j * VE;
            if (j < nvec) {
                if (edge(j)) {
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        if (inside(j, e)) Io<R>::st(out + e, r.get(e));
                } else {
                    r.store(out);
                }
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = r.get(e);
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = x.get(e);
        }
        if (edge(j)) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (!inside(j, e)) v[i][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) sum += v[i][e];
    }
    int n = G ? static_cast<int>(p.D) : warp_values<VE, NV>(nvec, w, T);
    if constexpr (SHIFT) {
        if (w == 0) n -= m;
        if (w == static_cast<int>((nvec - 1) % T) >> 5) n -= static_cast<int>(nvec * VE - m - p.D);
    }
    float mu = p.rms || n == 0 ? 0.0f : warp_sum<G ? G : 32>(sum) / static_cast<float>(n);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + static_cast<int64_t>(i) * T < nvec) {
            const int64_t j = t + static_cast<int64_t>(i) * T;
            if (edge(j)) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (inside(j, e)) sq = fmaf(v[i][e] - mu, v[i][e] - mu, sq);
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) sq = fmaf(v[i][e] - mu, v[i][e] - mu, sq);
            }
        }
    sq = warp_sum<G ? G : 32>(sq);
    const float inv_d = 1.0f / static_cast<float>(p.D);
    if constexpr (!G) {
        if (lane == 0) part[w] = make_float4(static_cast<float>(n), mu, sq, 0.0f);
        __syncthreads();
        // lane q takes warp q's part
        const float4 o = lane < (blockDim.x >> 5) ? part[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        mu = p.rms ? 0.0f : warp_sum(o.x * o.y) * inv_d;
        const float d = o.y - mu;
        sq = warp_sum(fmaf(o.x * d, d, o.z));
    }
    const float rstd = inv_sqrt(fmaf(sq, inv_d, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t j = t + static_cast<int64_t>(i) * T;
        if (j >= nvec) continue;
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] = (v[i][e] - mu) * rstd;
        auto column = [&](const float *of, float (&g)[VE]) {
            if constexpr (SHIFT) {
                weights_shifted(g, of, j * VE - m, p.D);
            } else {
                Raw<float, VE> q;
                q.load(of + j * VE);
#pragma unroll
                for (int e = 0; e < VE; ++e) g[e] = q.get(e);
            }
        };
        float g[VE];
        if (p.weight) {
            column(p.weight, g);
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] *= g[e];
        }
        if (p.bias) {
            column(p.bias, g);
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] += g[e];
        }
        IO *out = static_cast<IO *>(p.y) + at + j * VE;
        if (edge(j)) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (inside(j, e)) Io<IO>::st(out + e, v[i][e]);
            continue;
        }
        Raw<IO, VE> o;
        o.set(v[i]);
        o.store(out);
    }
    if (t == 0 && row < p.rows) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

// Rows of a ring: a group's, a block's, and a block's whose rows are so long that shared
// memory holds only one (4000 rows of 8192 fp32 values with a residual)
constexpr int kGroupStages = 4, kBlockStages = 2, kLongStages = 1;
// Threads of an SM: a thread's sums and its values of the row take about 100 registers
constexpr int kBwdThreads = 640;

// Bytes of a staged row: dy, s and (with DRES) dresidual
template <class IO, class R>
__host__ __device__ constexpr int64_t bwd_row_bytes(int64_t D, bool dres) {
    return D * (Io<IO>::kBytes + (dres ? 2 : 1) * Io<R>::kBytes);
}

// The pair with the halves that are off replaced by 0
__device__ __forceinline__ f2 and2(f2 v, bool lo, bool hi) {
    float a, b;
    unpack2(v, a, b);
    return pack2(lo ? a : 0.0f, hi ? b : 0.0f);
}

// A thread's NV VE values of a row as pairs, vector i at `at[i]` (in values), from memory or,
// without a row, from shared memory at `staged`.
template <class X, int VE, int NV>
__device__ __forceinline__ void load_pairs(const X *row, uint32_t staged, const int (&at)[NV],
                                           f2 (&v)[NV * VE / 2]) {
    Raw<X, VE> q[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (row == nullptr) q[i].load_shared(staged + at[i] * Io<X>::kBytes);
        else q[i].load(row + at[i]);
    }
#pragma unroll
    for (int k = 0; k < NV * VE / 2; ++k)
        v[k] = pack2(q[2 * k / VE].get(2 * k % VE), q[(2 * k + 1) / VE].get((2 * k + 1) % VE));
}

// IO: dy, dx; R: s, dresidual, ds.  G > 0: G lanes a row; G = 0: a block a row.  With VE > 1 the
// rows come through a ring in shared memory, filled by cp.async: every thread copies the
// vectors that it reads itself, so only its own copies are waited for.  Single values
// (VE = 1, rows of one warp) are loaded from memory; the warps of an SM cover each other there.  A thread's
// NV VE values are packed pairs: the pass would be bound by instructions otherwise.
// Dynamic shared memory: the weight (D floats; ones without a weight), then the rings, used
// again for the warps' sums (D floats each) at the end.
// SHIFT: the grid's rows are a multiple of VE apart, or a block has one row, so that m is the
// same for all of a block's rows and its columns stay where they are; D is then the width
// of the aligned vectors (Dp), the weight 0 in front of and behind the row.
template <class IO, class R, int VE, int NV, int G, int kStages, int SHIFT>
__global__ void __launch_bounds__(G ? 256 : kBwdThreads) norm_backward_kernel(const BwdParams p) {
    static_assert(!SHIFT || (G == 0 && VE > 1), "a block a row, by vectors");
    constexpr bool STAGED = VE > 1;
    constexpr int NP = NV * VE / 2;
    __shared__ float2 part[2][32];
    extern __shared__ __align__(16) unsigned char smem[];
    float *weight = reinterpret_cast<float *>(smem);
    const int m = SHIFT ? static_cast<int>(blockIdx.x * p.D % VE) : 0;
    const int64_t Dp = SHIFT ? (p.D + 2 * VE - 2) / VE * VE : p.D;
    unsigned char *ring = smem + (Dp * 4 + 15) / 16 * 16;
    float *columns = reinterpret_cast<float *>(ring);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int T = G ? G : blockDim.x, t = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
    const int groups = G ? blockDim.x / (G ? G : 1) : 1, group = G ? threadIdx.x / (G ? G : 1) : 0;
    const int nvec = static_cast<int>(SHIFT ? (p.D + m + VE - 1) / VE : p.D / VE);
    // this thread's vectors; in place of one past the row's end its first is read again (with
    // a weight of 0) and nothing is written; a thread without any only joins the sums
    int at[NV];
    bool live[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = t + i * T;
        live[i] = j < nvec;
        at[i] = (live[i] ? j : t) * VE;
    }
    auto edge = [&](int i) { return SHIFT && (at[i] == 0 || at[i] == (nvec - 1) * VE); };
    auto inside = [&](int i, int e) { return at[i] + e >= m && at[i] + e < p.D + m; };
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    // a warp's groups walk together (their sums are exchanged in one instruction): they end
    // when the warp's first row is past the last, and a row past it is empty
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
    const int64_t lead = G ? first - (threadIdx.x & 31) / (G ? G : 1) : first;
    const float inv_d = 1.0f / static_cast<float>(p.D);
    const uint32_t row_bytes = static_cast<uint32_t>(bwd_row_bytes<IO, R>(Dp, p.dresidual != nullptr));
    const uint32_t mine = smem_u32(ring) + group * kStages * row_bytes;
    const uint32_t off_s = static_cast<uint32_t>(Dp) * Io<IO>::kBytes, off_d = off_s + static_cast<uint32_t>(Dp) * Io<R>::kBytes;
    const bool dres = p.dresidual != nullptr;
    auto issue = [&](int64_t row, int stage) {
        if constexpr (STAGED) {
            if (row < p.rows) {
                const uint32_t to = mine + stage * row_bytes;
                const int64_t base = row * p.D - m;
                const char *gy = reinterpret_cast<const char *>(static_cast<const IO *>(p.dy) + base);
                const char *gs = reinterpret_cast<const char *>(static_cast<const R *>(p.s) + base);
                const char *gd = reinterpret_cast<const char *>(static_cast<const R *>(p.dresidual) + (dres ? base : 0));
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!live[i]) continue;
                    const uint32_t o = at[i] * Io<IO>::kBytes;
                    if constexpr (SHIFT) {
                        const int64_t left = p.rows * p.D - base - at[i];  // values to the tensor's end
                        if (left < VE) {
                            cp_async16_part(to + o, gy + o, static_cast<int>(left) * Io<IO>::kBytes);
                            for (int h = 0; h < VE * Io<R>::kBytes / 16; ++h) {
                                const int n = static_cast<int>(left) * Io<R>::kBytes - h * 16;
                                const uint32_t q = at[i] * Io<R>::kBytes + (n > 0 ? h * 16 : 0), z = off_s + at[i] * Io<R>::kBytes + h * 16;
                                cp_async16_part(to + z, gs + q, n > 16 ? 16 : n > 0 ? n : 0);
                                if (dres) cp_async16_part(to + z - off_s + off_d, gd + q, n > 16 ? 16 : n > 0 ? n : 0);
                            }
                            continue;
                        }
                    }
                    cp_async16(to + o, gy + o);
#pragma unroll
                    for (int h = 0; h < VE * Io<R>::kBytes / 16; ++h) {
                        const uint32_t q = at[i] * Io<R>::kBytes + h * 16;
                        cp_async16(to + off_s + q, gs + q);
                        if (dres) cp_async16(to + off_d + q, gd + q);
                    }
                }
            }
        }
        cp_async_commit();
    };
    if constexpr (SHIFT)
        for (int c = threadIdx.x; c < Dp; c += blockDim.x)
            if (c < m || c >= p.D + m) weight[c] = 0.0f;
    for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
        if (p.weight) cp_async4(weight + m + c, p.weight + c);
        else weight[m + c] = 1.0f;
    }
    cp_async_commit();
#pragma unroll
    for (int k = 0; k < kStages; ++k) issue(first + k * step, k);
    cp_async_wait<kStages>();  // the weight
    __syncthreads();
    f2 dw[NP], db[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) dw[k] = db[k] = 0;
    float mu = 0.0f, r = 0.0f;
    auto statistics = [&](int64_t row) {
        if (row < p.rows) mu = p.rms ? 0.0f : __ldg(p.mean + row), r = __ldg(p.rstd + row);
    };
    statistics(first);
    int par = 0, stage = 0;
    for (int64_t row = first, at0 = lead; at0 < p.rows; row += step, at0 += step, par ^= 1) {
        const bool work = live[0] && (!G || row < p.rows);
        const uint32_t from = mine + stage * row_bytes;
        if constexpr (STAGED) cp_async_wait<kStages - 1>();
        f2 z[NP], v[NP], a = 0, b = 0;
        const f2 mm = splat2(-mu), rr = splat2(r);
        if (work) {
            f2 wt[NP];
            load_pairs<R, VE, NV>(STAGED ? nullptr : static_cast<const R *>(p.s) + row * p.D, from + off_s, at, z);
            load_pairs<IO, VE, NV>(STAGED ? nullptr : static_cast<const IO *>(p.dy) + row * p.D, from, at, v);
            load_pairs<float, VE, NV>(nullptr, smem_u32(weight), at, wt);
            if constexpr (SHIFT) {  // other rows' values, which may be anything
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (edge(i)) {
#pragma unroll
                        for (int e = 0; e < VE; e += 2) {
                            const int k = (i * VE + e) / 2;
                            z[k] = and2(z[k], inside(i, e), inside(i, e + 1));
                            v[k] = and2(v[k], inside(i, e), inside(i, e + 1));
                        }
                    }
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                if (VE > 1 && !live[2 * k / VE]) wt[k] = 0;
                if (VE == 1) wt[k] = and2(wt[k], live[2 * k / VE], live[(2 * k + 1) / VE]);
                z[k] = mul2(add2(z[k], mm), rr);
                dw[k] = fma2(v[k], z[k], dw[k]);
                db[k] = add2(db[k], v[k]);
                v[k] = mul2(v[k], wt[k]);
                a = add2(a, v[k]);
                b = fma2(v[k], z[k], b);
            }
        }
        statistics(row + step);
        float s1, s2, hi;
        unpack2(a, s1, hi);
        s1 = warp_sum<G ? G : 32>(s1 + hi);
        unpack2(b, s2, hi);
        s2 = warp_sum<G ? G : 32>(s2 + hi);
        if constexpr (!G) {
            if (lane == 0) part[par][w] = make_float2(s1, s2);
            __syncthreads();  // the other half is written two rows on, after the next meeting
            const float2 o = lane < warps ? part[par][lane] : make_float2(0.0f, 0.0f);
            s1 = warp_sum(o.x);
            s2 = warp_sum(o.y);
        }
        const f2 m1 = splat2(p.rms ? 0.0f : -s1 * inv_d), m2 = splat2(-s2 * inv_d);
        if (work) {
            f2 d[NP];
            if (dres) {
                load_pairs<R, VE, NV>(STAGED ? nullptr : static_cast<const R *>(p.dresidual) + row * p.D, from + off_d, at, d);
            } else {
#pragma unroll
                for (int k = 0; k < NP; ++k) d[k] = 0;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float o[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const int k = (i * VE + e) / 2;
                    float lo, up;
                    unpack2(fma2(fma2(z[k], m2, add2(v[k], m1)), rr, d[k]), lo, up);
                    o[e] = (i * VE + e) & 1 ? up : lo;
                }
                if (!live[i]) continue;
                if (edge(i)) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        if (!inside(i, e)) continue;
                        Io<R>::st(static_cast<R *>(p.ds) + row * p.D - m + at[i] + e, o[e]);
                        if (p.dx) Io<IO>::st(static_cast<IO *>(p.dx) + row * p.D - m + at[i] + e, o[e]);
                    }
                    continue;
                }
                Raw<R, VE> q;
                q.set(o);
                q.store(static_cast<R *>(p.ds) + row * p.D - m + at[i]);
                if (p.dx) {
                    Raw<IO, VE> u;
                    u.set(o);
                    u.store(static_cast<IO *>(p.dx) + row * p.D - m + at[i]);
                }
            }
        }
        issue(row + kStages * step, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if constexpr (STAGED) cp_async_wait<0>();
    // the block's partial sums of the columns
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!(k == 0 ? p.want_dw : p.want_db)) continue;
        float *out = p.part + (static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * p.D;
        float *own = G ? columns + group * p.D : out;
        if constexpr (G) __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int c = (i * VE + e) / 2;
                float lo, up;
                unpack2(k == 0 ? dw[c] : db[c], lo, up);
                if (live[i] && (!SHIFT || inside(i, e))) own[at[i] + e - m] = (i * VE + e) & 1 ? up : lo;
            }
        }
        if constexpr (G) {
            __syncthreads();
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
                float sum = 0.0f;
                for (int q = 0; q < groups; ++q) sum += columns[q * p.D + c];
                out[c] = sum;
            }
        }
    }
}

// Rows too long for the registers of a block: one block a row, in several passes over it.  A
// thread takes NV vectors at a time (kLongValues values), so that a pass has them all in flight.
constexpr int kLongThreads = 512, kLongValues = 8;

// NV vectors of a row, vector j0 + i kLongThreads at i; past the row's end: zeros
template <class T, int VE, int NV>
__device__ __forceinline__ void load_long(Raw<T, VE> (&q)[NV], const T *row, int64_t j0, int64_t nvec) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t j = j0 + i * kLongThreads;
        q[i].zero();
        if (j < nvec) q[i].load(row + j * VE);
    }
}

// Sums of N values over the block, the same in every thread
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (&sm)[N][kLongThreads / 32]) {
#pragma unroll
    for (int q = 0; q < N; ++q) {
        v[q] = warp_sum(v[q]);
        if ((threadIdx.x & 31) == 0) sm[q][threadIdx.x >> 5] = v[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < N; ++q) {
        v[q] = 0.0f;
#pragma unroll
        for (int k = 0; k < kLongThreads / 32; ++k) v[q] += sm[q][k];
    }
    __syncthreads();
}

template <class IO, class R, bool RES, int VE>
__global__ void __launch_bounds__(kLongThreads) norm_forward_long_kernel(const FwdParams p) {
    constexpr int NV = kLongValues / VE;
    __shared__ float sm[1][kLongThreads / 32];
    const float inv_d = 1.0f / static_cast<float>(p.D);
    const int64_t row = blockIdx.x, nvec = p.D / VE;
    const IO *x = static_cast<const IO *>(p.x) + row * p.D;
    const R *r = RES ? static_cast<const R *>(p.residual) + row * p.D : nullptr;
    IO *y = static_cast<IO *>(p.y) + row * p.D;
    R *ro = RES ? static_cast<R *>(p.residual_out) + row * p.D : nullptr;
    // this thread's values of s from vector j0 on, rounded to R
    auto load = [&](int64_t j0, Raw<R, VE> (&s)[NV]) {
        Raw<IO, VE> a[NV];
        load_long(a, x, j0, nvec);
        if constexpr (RES) load_long(s, r, j0, nvec);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) v[e] = RES ? a[i].get(e) + s[i].get(e) : a[i].get(e);
            s[i].set(v);
        }
    };
    float v[1] = {0.0f};
    if (RES || !p.rms) {
        for (int64_t j0 = threadIdx.x; j0 < nvec; j0 += NV * kLongThreads) {
            Raw<R, VE> s[NV];
            load(j0, s);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t j = j0 + i * kLongThreads;
                if constexpr (RES)
                    if (j < nvec) s[i].store(ro + j * VE);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[0] += s[i].get(e);
            }
        }
    }
    float mu = 0.0f;
    if (!p.rms) {
        block_sums(v, sm);
        mu = v[0] * inv_d;
    }
    v[0] = 0.0f;
    for (int64_t j0 = threadIdx.x; j0 < nvec; j0 += NV * kLongThreads) {
        Raw<R, VE> s[NV];
        load(j0, s);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (j0 + i * kLongThreads < nvec) {
#pragma unroll
                for (int e = 0; e < VE; ++e) v[0] = fmaf(s[i].get(e) - mu, s[i].get(e) - mu, v[0]);
            }
    }
    block_sums(v, sm);
    const float rstd = inv_sqrt(v[0] * inv_d + p.eps);
    for (int64_t j0 = threadIdx.x; j0 < nvec; j0 += NV * kLongThreads) {
        Raw<R, VE> s[NV];
        Raw<float, VE> g[NV], b[NV];
        load(j0, s);
        if (p.weight) load_long(g, p.weight, j0, nvec);
        if (p.bias) load_long(b, p.bias, j0, nvec);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t j = j0 + i * kLongThreads;
            if (j >= nvec) continue;
            float o[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = (s[i].get(e) - mu) * rstd;
                if (p.weight) o[e] *= g[i].get(e);
                if (p.bias) o[e] += b[i].get(e);
            }
            Raw<IO, VE> u;
            u.set(o);
            u.store(y + j * VE);
        }
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mu;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

// Block k takes rows_per_block rows from k rows_per_block on, kLongRows at a time: their two
// sums, then the gradients with the rows read again (from the L2).  The columns' dw and db are
// kept in the block's own rows of part, each entry touched by one thread only; several rows
// at a time make that one read and write for all of them.  (3000 x 12288 bf16 106 us, one row
// and one value at a time 319; 2000 x 12288 fp32 132 and 277.)
constexpr int kLongRows = 4;
template <class IO, class R, int VE>
__global__ void __launch_bounds__(kLongThreads) norm_backward_long_kernel(const BwdParams p, int64_t rows_per_block) {
    constexpr int NV = kLongValues / VE, NR = kLongRows;
    __shared__ float sm[2 * NR][kLongThreads / 32];
    const float inv_d = 1.0f / static_cast<float>(p.D);
    float *pw = p.part + static_cast<int64_t>(blockIdx.x) * p.D;
    float *pb = p.part + (static_cast<int64_t>(gridDim.x) + blockIdx.x) * p.D;
    const int64_t nvec = p.D / VE, begin = blockIdx.x * rows_per_block;
    const int64_t end = begin + rows_per_block < p.rows ? begin + rows_per_block : p.rows;
    const bool dres = p.dresidual != nullptr;
    for (int64_t row0 = begin; row0 < end; row0 += NR) {
        const int n = end - row0 < NR ? static_cast<int>(end - row0) : NR;
        const IO *dy = static_cast<const IO *>(p.dy) + row0 * p.D;
        const R *s = static_cast<const R *>(p.s) + row0 * p.D;
        float mu[NR], rstd[NR], sums[2 * NR];
#pragma unroll
        for (int q = 0; q < NR; ++q) {
            mu[q] = p.rms || q >= n ? 0.0f : __ldg(p.mean + row0 + q);
            rstd[q] = q < n ? __ldg(p.rstd + row0 + q) : 0.0f;
            sums[2 * q] = sums[2 * q + 1] = 0.0f;
        }
        // the rows' values from vector j0 on (zeros of rows past the last), and the weight's
        Raw<R, VE> a[NR][NV];
        Raw<IO, VE> g[NR][NV];
        float w[NV][VE];
        auto load = [&](int64_t j0) {
#pragma unroll
            for (int q = 0; q < NR; ++q) {
                const int64_t count = q < n ? nvec : 0;
                load_long(a[q], s + q * p.D, j0, count);
                load_long(g[q], dy + q * p.D, j0, count);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                Raw<float, VE> t;
                t.zero();
                if (p.weight && j0 + i * kLongThreads < nvec) t.load(p.weight + (j0 + i * kLongThreads) * VE);
#pragma unroll
                for (int e = 0; e < VE; ++e) w[i][e] = p.weight ? t.get(e) : 1.0f;
            }
        };
        for (int64_t j0 = threadIdx.x; j0 < nvec; j0 += NV * kLongThreads) {
            load(j0);
#pragma unroll
            for (int q = 0; q < NR; ++q)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float v = g[q][i].get(e) * w[i][e];
                        sums[2 * q] += v;
                        sums[2 * q + 1] = fmaf(v, (a[q][i].get(e) - mu[q]) * rstd[q], sums[2 * q + 1]);
                    }
        }
        block_sums(sums, sm);
#pragma unroll
        for (int q = 0; q < NR; ++q) {
            sums[2 * q] = p.rms ? 0.0f : sums[2 * q] * inv_d;
            sums[2 * q + 1] *= inv_d;
        }
        for (int64_t j0 = threadIdx.x; j0 < nvec; j0 += NV * kLongThreads) {
            load(j0);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t j = j0 + i * kLongThreads;
                if (j >= nvec) continue;
                float dw[VE], db[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) dw[e] = db[e] = 0.0f;
#pragma unroll
                for (int q = 0; q < NR; ++q) {
                    if (q >= n) continue;
                    const int64_t at = (row0 + q) * p.D + j * VE;
                    Raw<R, VE> d;
                    if (dres) d.load(static_cast<const R *>(p.dresidual) + at);
                    float o[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float z = (a[q][i].get(e) - mu[q]) * rstd[q], v = g[q][i].get(e);
                        o[e] = rstd[q] * (v * w[i][e] - sums[2 * q] - z * sums[2 * q + 1]);
                        if (dres) o[e] += d.get(e);
                        dw[e] = fmaf(v, z, dw[e]);
                        db[e] += v;
                    }
                    Raw<R, VE> u;
                    u.set(o);
                    u.store(static_cast<R *>(p.ds) + at);
                    if (p.dx) {
                        Raw<IO, VE> t;
                        t.set(o);
                        t.store(static_cast<IO *>(p.dx) + at);
                    }
                }
                auto keep = [&](float *sum, const float (&v)[VE]) {
                    if constexpr (VE == 1) {
                        sum[j] = row0 == begin ? v[0] : sum[j] + v[0];
                    } else {
#pragma unroll
                        for (int e = 0; e < VE; e += 4) {
                            float4 *at = reinterpret_cast<float4 *>(sum + j * VE + e);
                            float4 o = row0 == begin ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *at;
                            o.x += v[e], o.y += v[e + 1], o.z += v[e + 2], o.w += v[e + 3];
                            *at = o;
                        }
                    }
                };
                if (p.want_dw) keep(pw, dw);
                if (p.want_db) keep(pb, db);
            }
        }
    }
}

}  // namespace norm
}  // namespace sscan
