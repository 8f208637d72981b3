// ssd_sum_rows.h -- sums over the rows of partial results in a fixed order.
#pragma once

#include "ssd_device.h"

namespace ssd {

// The sum of `rows` values (V: one or four floats) `stride` floats apart, for each of a 256-thread workgroup's 64
// lanes: four slices of the rows by a wave each, joined through LDS (256 values).  Every wave gets the sum.
template <typename V> __device__ inline V sum_rows(const float* src, int64_t stride, int rows, V* lds, bool live) {
    const int slice = threadIdx.x >> 6, lane = threadIdx.x & 63;
    V s = vzero<V>();
    if (live) {
#pragma unroll 8
        for (int r = slice; r < rows; r += 4) s += *(const V*)(src + r * stride);
    }
    lds[threadIdx.x] = s;
    __syncthreads();
    return (lds[lane] + lds[64 + lane]) + (lds[128 + lane] + lds[192 + lane]);
}

// The same for many rows of few values: 16 waves take a slice each (lds: 1024 values).
template <typename V> __device__ inline V sum_many_rows(const float* src, int64_t stride, int rows, V* lds, bool live) {
    const int slice = threadIdx.x >> 6, lane = threadIdx.x & 63;
    V s = vzero<V>();
    if (live) {
#pragma unroll 8
        for (int r = slice; r < rows; r += 16) s += *(const V*)(src + r * stride);
    }
    lds[threadIdx.x] = s;
    __syncthreads();
    V t = vzero<V>();
#pragma unroll
    for (int i = 0; i < 16; ++i) t += lds[i * 64 + lane];
    return t;
}

}  // namespace ssd
