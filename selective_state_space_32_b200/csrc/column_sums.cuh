// column_sums.cuh -- out[d] = sum_r part[r][d] in a fixed order (no atomics): the last
// step of every per-channel gradient (the recurrence's rate, the norm's weight and bias).
#pragma once

#include <cstdint>

namespace sscan {

constexpr int kColThreads = 256;  // 32 channels x 8 row lanes

// part [rows][D] fp32; grid.x = ceil(D / 32), grid.y = planes: plane k reads
// part + k * plane_stride and writes outs[k] (null: skipped).
struct ColumnSums {
    const float *part;
    float *out[2];
    int64_t rows, D, plane_stride;
};

static __global__ void __launch_bounds__(kColThreads) column_sums_kernel(const ColumnSums p) {
    __shared__ float sm[8][32];
    float *out = blockIdx.y == 0 ? p.out[0] : p.out[1];
    if (out == nullptr) return;  // the same for the whole block
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const float *part = p.part + blockIdx.y * p.plane_stride;
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
    if (d < p.D) {
        int64_t r = w;
        for (; r + 24 < p.rows; r += 32) {
            s0 += part[r * p.D + d];
            s1 += part[(r + 8) * p.D + d];
            s2 += part[(r + 16) * p.D + d];
            s3 += part[(r + 24) * p.D + d];
        }
        for (; r < p.rows; r += 8) s0 += part[r * p.D + d];
    }
    sm[w][lane] = (s0 + s1) + (s2 + s3);
    __syncthreads();
    if (w == 0 && d < p.D) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += sm[k][lane];
        out[d] = s;
    }
}

}  // namespace sscan
