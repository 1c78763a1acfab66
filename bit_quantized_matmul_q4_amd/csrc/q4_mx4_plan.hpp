// q4_mx4_plan.hpp -- sizes of the packed microscaled 4-bit form, and which
// kernel of its product a shape takes (host).  See q4_mx4.hip for the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace q4 {

// Steps of 128 k of a packed row tile, and groups of four of them.
__host__ __device__ inline int mx4_steps(int K) { return (K + 127) / 128; }
__host__ __device__ inline int mx4_groups(int K) { return (K + 511) / 512; }

// Where the codes of row, k .. k + 7 (k a multiple of 8), and the scale byte
// of the block that starts at k stand in the packed form.
__host__ __device__ inline size_t mx4_code_at(size_t row, int k, int K)
{
    return (row / 16 * mx4_steps(K) + k / 128) * 1024 + k / 32 % 4 * 256 + row % 16 * 16 + k % 32 / 2;
}
__host__ __device__ inline size_t mx4_scale_at(size_t row, int k, int K)
{
    return (row / 16 * mx4_groups(K) + k / 512) * 256 + k / 32 % 4 * 64 + row % 16 * 4 + k / 128 % 4;
}

// The tile of the product for a shape.
struct Mx4Shape {
    int bm, bn;
};

inline Mx4Shape mx4_shape(int M, int N, int K)
{
    (void)M, (void)N, (void)K;
    return Mx4Shape{64, 64};
}

}  // namespace q4
