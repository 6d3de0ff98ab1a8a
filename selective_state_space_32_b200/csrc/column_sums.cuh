// column_sums.cuh -- out[d] = sum_r part[r][d] in a fixed order (no atomics): the last
// step of every per-channel gradient (the recurrence's rate, the norm's weight and bias).
#pragma once

#include <cstdint>

namespace sscan {

constexpr int kColThreads = 1024;  // 32 channels x 32 row lanes

// part [rows][D] fp32; grid.x = ceil(D / 32), grid.y = planes: plane k reads
// part + k * plane_stride and writes outs[k] (null: skipped).
struct ColumnSums {
    const float *part;
    float *out[2];
    int64_t rows, D, plane_stride;
};

static __global__ void __launch_bounds__(kColThreads) column_sums_kernel(const ColumnSums p) {
    __shared__ float sm[32][33];
    float *out = blockIdx.y == 0 ? p.out[0] : p.out[1];
    if (out == nullptr) return;  // the same for the whole block
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const float *part = p.part + blockIdx.y * p.plane_stride;
    float a[8];  // eight loads in flight a thread: the kernel is a few rounds of latency
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = 0.0f;
    if (d < p.D) {
        for (int64_t r = w; r < p.rows; r += 256) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (r + 32 * k < p.rows) a[k] += part[(r + 32 * k) * p.D + d];
        }
    }
    sm[w][lane] = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
    __syncthreads();
    // warp w joins the 32 sums of channel w of the block's 32, by a tree
    float s = sm[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 32 + w;
    if (lane == 0 && e < p.D) out[e] = s;
}

}  // namespace sscan
