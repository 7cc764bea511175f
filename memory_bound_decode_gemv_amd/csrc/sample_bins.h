// sample_bins.h -- the sampler's bins: equal steps of m - x below a row's maximum
// m, over the part of the row's range that has weight.  Host and device code, so
// that the rule can be checked without a GPU.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>

namespace dg {

constexpr int kBins = 512;
constexpr float kLargestF32 = 3.4028234663852886e38f;

// m - x with infinities as the largest number: 0 where both are infinite.
__host__ __device__ __forceinline__ float bin_distance(float m, float x) {
    return fminf(fminf(m, kLargestF32) - fminf(x, kLargestF32), kLargestF32);
}

// Bins per unit of m - x.  low: the row's smallest value above -infinity; reach:
// the distance from which on an element has no weight.  The scale is never so
// small that the largest distance is ahead of the last bin: -infinity, with which
// the chunk kernels fill up a row's last load step, is in the last bin in every
// row.  Were it elsewhere, those places, which are behind the row, could be
// listed as candidates and read.
__host__ __device__ __forceinline__ float bin_scale(float m, float low, float reach) {
    if (m == INFINITY) return 1.0f;   // distances are 0 or the largest number
    const float range = fminf(fminf(m - low, reach), kLargestF32);
    return range > 0.0f ? fminf((float)kBins / range, 1e30f) : 1.0f;   // all alike: the distance is 0 at any scale
}

// The place among the bins: the bin is its integer part.  Larger for smaller x;
// equal values share a bin.
__host__ __device__ __forceinline__ float bin_place(float distance, float scale) {
    return fminf(distance * scale, (float)(kBins - 1));
}

}  // namespace dg
