// kernel_glr_scan.cuh -- the gated linear recurrence over a sequence, parallel along it.
//
// A token is the affine map h -> a h + b, and maps compose: (a2, b2) after (a1, b1) is
// (a1 a2, a2 b1 + b2).  A warp owns a run of K tokens of kRowBytes = 128 bytes of
// channels (64 in bf16, two a lane; 32 in fp32), a block W consecutive runs, a cluster
// of C blocks C W consecutive runs, and the cluster walks the sequence of one batch row
// and channel group in steps of C W runs:
//   1. every warp computes a and b of its run (registers) and the run's composition;
//   2. the block's warps exchange compositions through shared memory, and the cluster's
//      blocks the blocks' through distributed shared memory;
//   3. every thread applies what precedes its run to the carried state, walks its
//      tokens once more and stores them; the carried state moves on by the composition
//      of the whole step, which every block forms for itself in the same order.
// So x and the gates are read once, y is written once, and the order of the sums depends on the
// sizes only.  Only drate's partial sums go through a workspace.  The blocks of a cluster wait for
// each other's maps on mbarriers in shared memory, for a bounded time; the blocks of different
// clusters do not wait.  The next steps' inputs arrive by cp.async in a ring of each warp's own
// while this one runs.
// The backward pass is the same walk from the last token: G_t = dy_t + e, e <- a_t G_t is
// a map of e, with the states of a run recomputed from the saved state before it.
//
// What bounds it (B200).  fp32 is a stream: 8 x 2048 x 1536 without a rate 49 us, 95 % of the
// copy rate.  bf16 moves half the bytes and waits: with a rate and an input gate 39 instructions
// a value forward, of which 19 on the FMA pipe and 4 on the MUFU (53 us for 8 x 2048 x 1536,
// 59 % of the copy rate), 70 backward (104 us, 54 %); issue is 58 and 52 % busy, no pipe above
// 50 %, and the 9.6 warps of an SM spend their time on fixed latencies (0.9 of 2.1 and 1.0 of 2.8
// stall cycles an instruction) and on memory and the cluster's maps (0.5 and 0.9).  Without rate
// and input gate 72 and 154 us for 2 x 8192 x 4096 (86 and 71 %).  A few long walks wait for their
// exchanges: 1 x 131072 x 2048 602 us (55 %).
//
// Runs of 16 tokens halve the exchanges of runs of 8 (67 against 74 us for the first bf16
// case); the backward pass would not fit its registers with them.  Maps by st.async instead of
// plain stores and a cluster barrier, which has to fence every thread's output stores: 65 ->
// 59 us for that case, backward 135 -> 113.
//
// Tokens past the end of a sequence get, in shared memory, the gate that makes their map the
// identity, so that the arithmetic has no case for them (selects in registers: 78 against 73 us
// for 2 x 8192 x 4096).
//
// Rows that are not a multiple of 16 bytes cannot be copied by cp.async 16 bytes at a
// time; STAGED = false loads them from memory, one channel a lane.
#pragma once

#include "cp_async.cuh"
#include "device_utils.cuh"
#include "glr_math.cuh"
#include "kernel_glr.cuh"

namespace sscan {
namespace glr {

constexpr int kMaxWarps = 8;
constexpr int kMaxCluster = 16;  // above 8 is not portable between devices; this one has 16
constexpr int kStages = 2;
constexpr int kForwardRun = 16;  // tokens of a warp's run; the backward pass takes kRun (a saved state each)

// Channels a lane holds: a pair where rows are staged in bf16, or one.  (One channel a lane in
// bf16 too, 64 bytes a row, measured slower wherever there is work to fill the device: 192
// chains of 2048 tokens 59 us against 53, 128 of 8192 109 against 78, 32 of 131072 745
// against 621; faster for a single chain of 65536 only, 71 against 94.)
template <class IO, bool STAGED> constexpr int lane_channels() { return STAGED ? 4 / Io<IO>::kBytes : 1; }
// Blocks of kMaxWarps an SM holds.  One channel a lane: 80 registers, three (384 fp32 chains
// of 2048 tokens, backward: 89 us, with two blocks 106; odd widths, 2 x 3000 x 1201 fp32 with
// both gates, 32 and 60 us, with two 40 and 79); two: 128, since 80 would spill (bf16 with rate
// and input gate, 192 chains, backward: two blocks 103 us, three 113).
template <int V> constexpr int scan_blocks() { return V == 1 ? 3 : 2; }

// Bytes of a staged row: the channels of a warp
template <class IO, int V> constexpr int row_bytes() { return 32 * V * Io<IO>::kBytes; }

template <class IO, int V, bool STAGED, int NS, int K>
constexpr int scan_smem_bytes(int warps, int cluster) {
    return 128 + (STAGED ? warps * kStages * NS * K * row_bytes<IO, V>() : 0) + 2 * (warps + cluster) * 32 * V * 8;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The warp's index, known to the compiler to be the same in its lanes (row addresses are
// then formed once a warp)
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }

// A lane's V channels: one value, or a packed pair.
template <int V> struct Lane;
template <> struct Lane<1> {
    using T = float;
    static __device__ __forceinline__ float mul(float a, float b) { return a * b; }
    static __device__ __forceinline__ float add(float a, float b) { return a + b; }
    static __device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
    static __device__ __forceinline__ float splat(float v) { return v; }
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
    // token k of an array of pairs: half k % 2 of pair k / 2
    template <int NP> static __device__ __forceinline__ float get(const f2 (&v)[NP], int k) {
        float a, b;
        unpack2(v[k / 2], a, b);
        return k & 1 ? b : a;
    }
};
template <> struct Lane<2> {
    using T = f2;
    static __device__ __forceinline__ f2 mul(f2 a, f2 b) { return mul2(a, b); }
    static __device__ __forceinline__ f2 add(f2 a, f2 b) { return add2(a, b); }
    static __device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) { return fma2(a, b, c); }
    static __device__ __forceinline__ f2 splat(float v) { return splat2(v); }
    static __device__ __forceinline__ f2 load(const float *p) { return pack2(p[0], p[1]); }
    static __device__ __forceinline__ void store(float *p, f2 v) { store_channels<float, 2>(p, v); }
    // token k of an array of pairs: pair k
    template <int NP> static __device__ __forceinline__ f2 get(const f2 (&v)[NP], int k) { return v[k]; }
};
template <class IO> __device__ __forceinline__ void store_lane(IO *p, float v) { Io<IO>::st(p, v); }
template <class IO> __device__ __forceinline__ void store_lane(IO *p, f2 v) { store_channels<IO, 2>(p, v); }

// One warp's view of its streams: NS tensors [B][L][D] in runs of K tokens, and a lane's
// V channels of them as pairs (V = 2: the channels of one token; V = 1: two tokens).
template <class IO, int V, bool STAGED, int NS, int K>
struct RunLoader {
    static constexpr int CH = 32 * V, NP = K * V / 2;
    static constexpr int kRowBytes = row_bytes<IO, V>(), kStageBytes = NS * K * kRowBytes;
    static constexpr int kRowLanes = kRowBytes / 16, kRows = 32 / kRowLanes;  // lanes that copy a row, rows at once
    const IO *src[NS];  // batch row's first token, first channel of the group
    unsigned char *ring;
    int64_t L, D;
    int lane, live;  // live: channels of the group that exist

    // Start copying the run of tokens t0 .. t0 + K - 1 at `off` = t0 D values (tokens past L,
    // channels past D: zeros).
    __device__ __forceinline__ void issue(int64_t t0, int64_t off, int stage) const {
        if constexpr (STAGED) {
            if (t0 >= 0 && t0 < L) {
                const int at16 = lane % kRowLanes, col = at16 * (16 / Io<IO>::kBytes), row = lane / kRowLanes;
                const uint32_t own = row * static_cast<uint32_t>(D) + col;  // under 8 rows of 2^28 channels
                const int64_t next = kRows * D;
                unsigned char *dst = ring + stage * kStageBytes + row * kRowBytes + at16 * 16;
                if (live == CH && t0 + K <= L) {
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const IO *p = src[s] + off;
#pragma unroll
                        for (int h = 0; h < K / kRows; ++h, p += next)
                            cp_async16(dst + (s * K + kRows * h) * kRowBytes, p + own);
                    }
                } else {
                    const int n = col < live ? (L - t0 < K ? static_cast<int>(L - t0) : K) : 0;
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int h = 0; h < K / kRows; ++h)
                            cp_async16_part(smem_u32(dst + (s * K + kRows * h) * kRowBytes),
                                            row + kRows * h < n ? src[s] + off + h * next + own : src[s],
                                            row + kRows * h < n ? 16 : 0);
                }
            }
            cp_async_commit();
        }
    }
    // Tokens past the end of a run of n: zeros, and in stream 1, the gate, the value that makes
    // the token's map the identity.  Every lane writes what it will read itself.
    __device__ __forceinline__ void pad(int n, int stage, float gate) const {
        if constexpr (STAGED) {
            IO *at = reinterpret_cast<IO *>(ring + stage * kStageBytes) + lane * V;
            for (int k = n; k < K; ++k)
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int j = 0; j < V; ++j) Io<IO>::st(at + (s * K + k) * CH + j, s == 1 ? gate : 0.0f);
        }
    }
    // stream s, pair i of the run at t0 with n tokens (not staged: `past` for those past the end)
    __device__ __forceinline__ f2 pair(int64_t t0, int n, int stage, int s, int i, float past) const {
        if constexpr (STAGED) {
            const unsigned char *at = ring + stage * kStageBytes + s * K * kRowBytes;
            if constexpr (V == 2) {
                const uint32_t v = reinterpret_cast<const uint32_t *>(at)[i * 32 + lane];
                return pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
            } else {
                const IO *w = reinterpret_cast<const IO *>(at) + lane;
                return pack2(Io<IO>::widen(w[2 * i * 32]), Io<IO>::widen(w[(2 * i + 1) * 32]));
            }
        } else {
            const IO *p = src[s] + (t0 + 2 * i) * D + lane;
            const bool on = lane < live;
            return pack2(on && 2 * i < n ? Io<IO>::widen(Io<IO>::ld(p)) : past,
                         on && 2 * i + 1 < n ? Io<IO>::widen(Io<IO>::ld(p + D)) : past);
        }
    }
};

// The gate of a token whose map is the identity: a = 1 and beta = 0
template <bool DECAY> __device__ __forceinline__ float idle_gate() { return __uint_as_float(DECAY ? 0xff800000u : 0x7f800000u); }

// (decay, offset) of one lane's channels in shared memory: V * 8 bytes
__device__ __forceinline__ void load_map(const float2 *p, float &a, float &h) {
    const float2 m = *p;
    a = m.x, h = m.y;
}
__device__ __forceinline__ void load_map(const float2 *p, f2 &a, f2 &h) {
    const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(p);
    a = m.x, h = m.y;
}
__device__ __forceinline__ void store_map(float2 *p, float a, float h) { *p = make_float2(a, h); }
__device__ __forceinline__ void store_map(float2 *p, f2 a, f2 h) {
    *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(a, h);
}
// The address that `local` (shared memory of this block) has in block `rank`.
__device__ __forceinline__ uint32_t cluster_address(const void *local, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
    return at;
}
// Store a lane's maps there; their bytes are counted on that block's mbarrier.  (A cluster
// barrier instead has to fence every thread's earlier stores of outputs first.)
__device__ __forceinline__ void send_map(float2 *local, uint64_t *bar, uint32_t rank, float a, float h) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                     cluster_address(local, rank)), "f"(a), "f"(h), "r"(cluster_address(bar, rank))
                 : "memory");
}
__device__ __forceinline__ void send_map(float2 *local, uint64_t *bar, uint32_t rank, f2 a, f2 h) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(
                     cluster_address(local, rank)), "l"(a), "l"(h), "r"(cluster_address(bar, rank))
                 : "memory");
}
// mbar_wait for bytes that other blocks of the cluster stored
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, uint32_t tries) {
    for (uint32_t i = 0; i < tries; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}

// The waits of a cluster's blocks for one another: how often each looks before it gives up,
// and the caller's word (or null) that is told of it.  An argument of its own: as a part of
// FwdParams it made the launch of the step kernel, which has no waits, 0.7 us longer.
struct Waits {
    int *status;
    uint32_t tries;
};
constexpr int kGaveUp = 1;  // the bit set in *status

// What the blocks and warps of a cluster share in a walk: agg [2][warps][CH] and
// cl [2][C][CH] maps and two mbarriers, used in turn by the steps.  A step's entries are
// overwritten two steps later: by then this block's warps have met at the step between
// them, and a block sends its second next maps only after it has this block's next ones,
// which this block's warps send after that meeting.
struct Shared {
    float2 *agg, *cl;
    uint64_t *bar;
    uint32_t C, rank;
    int warps, w, lane;
    Waits waits;
    // A wait for the cluster's maps gave up (1 + the step's low two bits): the state is NaN from
    // there on, and this thread sends and arms no more, so that the other blocks' waits give up
    // too, once each.
    int lost;

    // reads: have_read will follow
    __device__ __forceinline__ void init(unsigned char *smem, unsigned char *maps, int ch, uint32_t cluster,
                                         const Waits &wt, bool reads = false) {
        C = cluster;
        waits = wt;
        rank = C > 1 ? cluster_rank() : 0;
        lane = threadIdx.x & 31, w = warp_index(), warps = blockDim.x >> 5;
        bar = reinterpret_cast<uint64_t *>(smem);
        agg = reinterpret_cast<float2 *>(maps);
        cl = agg + 2 * warps * ch;
        lost = 0;
        if (C > 1) {
            if (threadIdx.x == 0) {
                for (int k = 0; k < 2; ++k) mbar_init(bar + k, 1), mbar_expect_tx(bar + k, C * ch * 8);
                mbar_fence_init();
            }
            __syncwarp();
            if (!reads) cluster_arrive();
        }
    }
    // Once the caller has read the initial state that another block overwrites at the end.
    __device__ __forceinline__ void have_read() const {
        __syncwarp();
        if (C > 1) cluster_arrive();
    }
    // Every block of the cluster has set up its mbarriers: it may be sent to.
    __device__ __forceinline__ void start() const {
        __syncwarp();
        if (C > 1) cluster_wait();
    }
    // The wait of step `it` gave up (finish reports it: an atomic here instead, in the walk's
    // loop, made the directly loaded bf16 backward 6 % slower).
    __device__ __forceinline__ void give_up(int64_t it) { lost = 1 + static_cast<int>(it & 3); }
    // A thread that lost a wait stays until what the others had sent for that step has arrived
    // (for a bounded time: they may not have), and until they have come here or ended: till then
    // they may still send to its block.  What a block sends later than that step, it sends
    // before a wait of its own that gives up.
    __device__ __forceinline__ void finish() const {
        if (lost) {
            if (waits.status) atomicOr(waits.status, kGaveUp);
            mbar_wait_sleep(bar + (lost - 1 & 1), static_cast<uint32_t>(lost - 1 >> 1));
            asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
        }
    }
};

// The exchange of step `it`.  In: the composition (A, H) of this warp's run, the state
// `carry` before the step.  Returns the state before the run; `carry` becomes the state
// after the step.
template <int V>
__device__ __forceinline__ typename Lane<V>::T exchange(typename Lane<V>::T A, typename Lane<V>::T H,
                                                        typename Lane<V>::T &carry, Shared &sh, int64_t it) {
    using LV = Lane<V>;
    using T = typename LV::T;
    constexpr int CH = 32 * V;
    const int par = static_cast<int>(it & 1), w = sh.w, warps = sh.warps;
    const float2 *at = sh.agg + par * warps * CH + sh.lane * V;
    __syncwarp();
    if (warps > 1) {
        store_map(sh.agg + (par * warps + w) * CH + sh.lane * V, A, H);
        __syncthreads();
    }
    if (sh.C == 1) {
        if (warps == 1) {
            const T h = carry;
            carry = LV::fma(A, carry, H);
            return h;
        }
        T h = carry;
#pragma unroll 2
        for (int q = 0; q < warps; ++q, at += CH) {
            T ma, mh;
            load_map(at, ma, mh);
            if (q == w) h = carry;
            carry = LV::fma(ma, carry, mh);
        }
        return h;
    }
    // the runs of this block before this one; the warps that send go on to the whole block
    T Ab = LV::splat(1.0f), Hb = LV::splat(0.0f);
    int q = 0;
#pragma unroll 2
    for (; q < w; ++q, at += CH) {
        T ma, mh;
        load_map(at, ma, mh);
        Ab = LV::mul(ma, Ab);
        Hb = LV::fma(ma, Hb, mh);
    }
    const T Ap = Ab, Hp = Hb;
    if (static_cast<uint32_t>(w) < sh.C && !sh.lost) {
        if (warps == 1) {
            Ab = A, Hb = H;
        } else {
#pragma unroll 2
            for (; q < warps; ++q, at += CH) {
                T ma, mh;
                load_map(at, ma, mh);
                Ab = LV::mul(ma, Ab);
                Hb = LV::fma(ma, Hb, mh);
            }
        }
        for (uint32_t r = w; r < sh.C; r += warps)
            send_map(sh.cl + (par * sh.C + sh.rank) * CH + sh.lane * V, sh.bar + par, r, Ab, Hb);
    }
    if (!sh.lost && !mbar_wait_cluster(sh.bar + par, static_cast<uint32_t>(it >> 1) & 1, sh.waits.tries)) {
        sh.give_up(it);
        carry = LV::splat(__uint_as_float(0x7fc00000u));
    }
    if (threadIdx.x == 0 && !sh.lost) mbar_expect_tx(sh.bar + par, sh.C * CH * 8);  // for the second next step
    at = sh.cl + par * sh.C * CH + sh.lane * V;
    T h = carry;
#pragma unroll 2
    for (uint32_t r = 0; r < sh.C; ++r, at += CH) {
        T ma, mh;
        load_map(at, ma, mh);
        if (r == sh.rank) h = carry;
        carry = LV::fma(ma, carry, mh);
    }
    return LV::fma(Ap, h, Hp);
}

// grid: B * groups * C blocks of 32 W threads in clusters of C
template <class IO, int V, bool STAGED, bool DECAY, bool IG, int K>
__global__ void __launch_bounds__(32 * kMaxWarps, scan_blocks<V>())
glr_scan_kernel(const FwdParams p, const Waits waits, int64_t groups, uint32_t C) {
    constexpr int NS = IG ? 3 : 2;
    using Loader = RunLoader<IO, V, STAGED, NS, K>;
    constexpr int CH = Loader::CH, NP = Loader::NP;
    using LV = Lane<V>;
    using T = typename LV::T;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, w = warp_index(), warps = blockDim.x >> 5;
    Shared sh;
    const bool in_place = p.h0 && p.h_final == p.h0;
    sh.init(smem, smem + 128 + (STAGED ? warps * kStages * Loader::kStageBytes : 0), CH, C, waits, in_place);
    const uint32_t rank = sh.rank;
    const int64_t cid = blockIdx.x / C, b = cid / groups, ch0 = (cid - b * groups) * CH;
    const int64_t row0 = b * p.L * p.D + ch0;
    Loader in;
    in.src[0] = static_cast<const IO *>(p.x) + row0;
    in.src[1] = static_cast<const IO *>(p.gate) + row0;
    if constexpr (IG) in.src[2] = static_cast<const IO *>(p.igate) + row0;
    in.ring = smem + 128 + w * kStages * Loader::kStageBytes;
    in.L = p.L, in.D = p.D, in.lane = lane;
    in.live = static_cast<int>(p.D - ch0 < CH ? p.D - ch0 : CH);
    const int64_t step = static_cast<int64_t>(C) * warps * K;  // tokens
    int64_t t0 = (static_cast<int64_t>(rank) * warps + w) * K;
    const int64_t steps = (p.L + step - 1) / step, pitch = step * p.D;
    int64_t off = t0 * p.D;
#pragma unroll
    for (int s = 0; s < kStages; ++s) in.issue(t0 + s * step, off + s * pitch, s);
    const bool mine = lane * V < in.live;
    T carry = LV::splat(0.0f);
    f2 cc = 0;  // rate log2 e of the pair
    if (mine) {
        if constexpr (DECAY) cc = mul2(capped_rate(load_channels<float, V>(p.rate + ch0 + lane * V)), splat2(kLog2e));
        if (p.h0) carry = LV::load(p.h0 + b * p.D + ch0 + lane * V);
    }
    if (in_place) sh.have_read();
    IO *y = static_cast<IO *>(p.y) + row0;
    const uint32_t own = lane * V;
    float *states = p.states ? p.states + b * p.nruns * p.D + ch0 : nullptr;
    sh.start();
    int stage = 0;
    for (int64_t it = 0; it < steps; ++it, t0 += step, off += pitch) {
        const int n = t0 >= p.L ? 0 : p.L - t0 < K ? static_cast<int>(p.L - t0) : K;
        f2 a[NP], bb[NP];
        if constexpr (STAGED) {
            cp_async_wait<kStages - 1>();
            __syncwarp();
        }
        if (n < K) in.pad(n, stage, idle_gate<DECAY>());
#pragma unroll
        for (int i = 0; i < NP; ++i)
            token2<DECAY, IG>(in.pair(t0, n, stage, 0, i, 0.0f), in.pair(t0, n, stage, 1, i, idle_gate<DECAY>()),
                              IG ? in.pair(t0, n, stage, NS - 1, i, 0.0f) : 0, cc, a[i], bb[i]);
        T A = LV::get(a, 0), H = LV::get(bb, 0);
#pragma unroll
        for (int k = 1; k < K; ++k) {
            A = LV::mul(A, LV::get(a, k));
            H = LV::fma(LV::get(a, k), H, LV::get(bb, k));
        }
        __syncwarp();
        in.issue(t0 + kStages * step, off + kStages * pitch, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        T h = exchange<V>(A, H, carry, sh, it);
        IO *yt = y + off;
        auto emit = [&](int k) {
            if (k % kRun == 0 && states) LV::store(states + off / kRun + k / kRun * p.D + own, h);
            h = LV::fma(LV::get(a, k), h, LV::get(bb, k));
            store_lane<IO>(yt + own, h);
            yt += p.D;
        };
        if (mine && n == K) {
#pragma unroll
            for (int k = 0; k < K; ++k) emit(k);
        } else if (mine) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (k < n) emit(k);
        }
    }
    if (p.h_final && rank == 0 && w == 0 && mine) LV::store(p.h_final + b * p.D + ch0 + lane * V, carry);
    sh.finish();
}

// The walk from the last token.  part (with a rate): row b * C + rank holds the sums of
// this block's channels.
template <class IO, int V, bool STAGED, bool DECAY, bool IG>
__global__ void __launch_bounds__(32 * kMaxWarps, scan_blocks<V>())
glr_scan_backward_kernel(const BwdParams p, const Waits waits, int64_t groups, uint32_t C) {
    constexpr int NS = IG ? 4 : 3, K = kRun;
    using Loader = RunLoader<IO, V, STAGED, NS, K>;
    constexpr int CH = Loader::CH, NP = Loader::NP;
    using LV = Lane<V>;
    using T = typename LV::T;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, w = warp_index(), warps = blockDim.x >> 5;
    Shared sh;
    sh.init(smem, smem + 128 + (STAGED ? warps * kStages * Loader::kStageBytes : 0), CH, C, waits);
    const uint32_t rank = sh.rank;
    const int64_t cid = blockIdx.x / C, b = cid / groups, ch0 = (cid - b * groups) * CH;
    const int64_t row0 = b * p.L * p.D + ch0;
    Loader in;
    in.src[0] = static_cast<const IO *>(p.x) + row0;
    in.src[1] = static_cast<const IO *>(p.gate) + row0;
    in.src[2] = static_cast<const IO *>(p.dy) + row0;
    if constexpr (IG) in.src[3] = static_cast<const IO *>(p.igate) + row0;
    in.ring = smem + 128 + w * kStages * Loader::kStageBytes;
    in.L = p.L, in.D = p.D, in.lane = lane;
    in.live = static_cast<int>(p.D - ch0 < CH ? p.D - ch0 : CH);
    const int64_t step = static_cast<int64_t>(C) * warps * K;  // tokens
    int64_t t0 = (p.nruns - 1 - (static_cast<int64_t>(rank) * warps + w)) * K;  // this warp's run of the first step
    const int64_t steps = (p.nruns * K + step - 1) / step, pitch = step * p.D;
    int64_t off = t0 * p.D;
#pragma unroll
    for (int s = 0; s < kStages; ++s) in.issue(t0 - s * step, off - s * pitch, s);
    const bool mine = lane * V < in.live;
    T carry = LV::splat(0.0f), dc = LV::splat(0.0f);
    f2 cn = 0, cl2 = 0;  // the pair's rate, and rate log2 e
    if (mine) {
        if constexpr (DECAY) {
            cn = capped_rate(load_channels<float, V>(p.rate + ch0 + lane * V));
            cl2 = mul2(cn, splat2(kLog2e));
        }
        if (p.dh_final) carry = LV::load(p.dh_final + b * p.D + ch0 + lane * V);
    }
    const uint32_t own = lane * V;
    const float *states = p.states + b * p.nruns * p.D + ch0 + own;
    sh.start();
    int stage = 0;
    for (int64_t it = 0; it < steps; ++it, t0 -= step, off -= pitch) {
        const int n = t0 < 0 ? 0 : p.L - t0 < K ? static_cast<int>(p.L - t0) : K;
        f2 a[NP], g[NP], px[NP], pi[NP], pg[NP], pr[NP];
        T h = LV::splat(0.0f);
        if (mine && n > 0) h = LV::load(states + off / K);
        if constexpr (STAGED) {
            cp_async_wait<kStages - 1>();
            __syncwarp();
        }
        if (n < K) in.pad(n, stage, idle_gate<DECAY>());
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            f2 bb, v, kg, kr, d;
            g[i] = in.pair(t0, n, stage, 2, i, 0.0f);
            token_grad2<DECAY, IG>(in.pair(t0, n, stage, 0, i, 0.0f), in.pair(t0, n, stage, 1, i, idle_gate<DECAY>()),
                                   IG ? in.pair(t0, n, stage, NS - 1, i, 0.0f) : 0, cn, cl2, a[i], bb, v, px[i], pi[i], kg, kr);
            if constexpr (V == 2) {
                d = minus2(v, h);
                h = fma2(a[i], h, bb);
            } else {  // two tokens of one channel: the second's state follows from the first's
                float a0, a1, b0, b1;
                unpack2(a[i], a0, a1);
                unpack2(bb, b0, b1);
                const float h1 = fmaf(a0, h, b0);
                d = minus2(v, pack2(h, h1));
                h = fmaf(a1, h1, b1);
            }
            pg[i] = mul2(kg, d);
            pr[i] = mul2(kr, d);
        }
        T A = LV::splat(1.0f), F = LV::splat(0.0f);
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {  // e -> a (g + e), last token first
            F = LV::mul(LV::get(a, k), LV::add(LV::get(g, k), F));
            A = LV::mul(A, LV::get(a, k));
        }
        __syncwarp();
        in.issue(t0 - kStages * step, off - kStages * pitch, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        T e = exchange<V>(A, F, carry, sh, it);
        const int64_t at = row0 + off;
        IO *dx = static_cast<IO *>(p.dx) + at, *dg = static_cast<IO *>(p.dgate) + at;
        IO *di = IG ? static_cast<IO *>(p.digate) + at : nullptr;
        auto emit = [&](int k) {
            const T G = LV::add(LV::get(g, k), e);
            e = LV::mul(LV::get(a, k), G);
            if constexpr (DECAY) dc = LV::fma(G, LV::get(pr, k), dc);
            store_lane<IO>(dx + k * p.D + own, LV::mul(G, LV::get(px, k)));
            store_lane<IO>(dg + k * p.D + own, LV::mul(G, LV::get(pg, k)));
            if constexpr (IG) store_lane<IO>(di + k * p.D + own, LV::mul(G, LV::get(pi, k)));
        };
        if (mine && n == K) {
#pragma unroll
            for (int k = K - 1; k >= 0; --k) emit(k);
        } else if (mine) {
#pragma unroll
            for (int k = K - 1; k >= 0; --k)
                if (k < n) emit(k);
        }
    }
    if (p.dh0 && rank == 0 && w == 0 && mine) LV::store(p.dh0 + b * p.D + ch0 + lane * V, carry);
    if constexpr (DECAY) {
        float *sums = reinterpret_cast<float *>(sh.agg);  // [warps][CH], once the last step's entries are read
        __syncthreads();
        LV::store(sums + w * CH + lane * V, dc);
        __syncthreads();
        if (w == 0 && mine) {
            for (int q = 1; q < warps; ++q) dc = LV::add(dc, LV::load(sums + q * CH + lane * V));
            LV::store(p.part + (b * C + rank) * p.D + ch0 + lane * V, dc);
        }
    }
    sh.finish();
}

}  // namespace glr
}  // namespace sscan
