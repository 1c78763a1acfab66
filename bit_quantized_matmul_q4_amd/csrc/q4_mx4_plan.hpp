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

constexpr int kMx4Units = 256;  // compute units

// Bytes of LDS that few rows take.
__host__ __device__ constexpr int mx4_few_lds(int M, int K)
{
    return M * ((K + 127) / 128 * 64 + (K + 511) / 512 * 16);
}

// The kernels of the product: two for few rows, tiles of rows x columns for more.
enum class Mx4Kernel { relay, wide, tile16x32, tile32x32, tile32x64, tile64x64, tile64x128, tile128x128, tile128x256 };

struct Mx4Shape {
    bool fused;  // dense rows are quantized within the product
    Mx4Kernel kernel;
};

inline long long mx4_tile_count(int M, int N, int bm, int bn)
{
    return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

inline Mx4Shape mx4_shape(bool dense, int M, int N, int K)
{
    // Quantizing within the product saves a launch, and every workgroup does it
    // again: us fused / apart at 3584 x 3584, 1 / 2 / 4 / 8 rows 5.0 / 5.3 / 6.3 /
    // 8.2 against 7.1; 896 x 896, 1 / 8 / 16 rows 3.2 / 3.7 / 4.6 against 5.2; 3584 x
    // 18944 at one row 15.9 against 14.3.
    if (M <= 16) {
        Mx4Shape s{dense && M * K <= 14336, Mx4Kernel::relay};
        // A wave a tile of 16 columns, where every wave has one (us, relay / wide):
        // 18944 x 3584 at 1 / 4 rows 10.5 / 10.8, 14.2 / 13.0; 152064 x 896 27.8 /
        // 15.0; 3584 x 3584 5.0 / 5.5.  A run of steps that holds all of K leaves the
        // relay one wave: 4864 x 896 4.0 / 3.3.
        const bool fits = mx4_few_lds(M, K) <= 60 * 1024;
        if (fits && (N >= 16384 || mx4_steps(K) <= 8))
            s.kernel = Mx4Kernel::wide;
        return s;
    }
    // The largest tile whose workgroups still fill more than half of the card, and
    // whose rows are not mostly padding.  Measured (us on packed rows, 128 x 256 /
    // 128 x 128 / 64 x 128 / 64 x 64 / 32 x 64 / 32 x 32 / 16 x 32):
    //   512 x 18944 x 3584  32.5 / 40.8 / 39.7 / 49.4 / 62.0 / 69.2 / 90.8
    //   200 x 18944 x 3584  20.1 / 27.1 / 23.2 / 31.1 / 29.3 / 35.3 / 45.4
    //   1024 x 3584 x 3584  16.4 / 14.4 / 14.9 / 22.7 / 21.6 / 26.5 / 37.0
    //   124 x 18944 x 3584  20.4 / 16.5 / 19.6 / 18.7 / 20.8 / 23.7 / 31.0
    //   4000 x 896 x 896    11.0 /  8.4 /  7.7 / 13.8 /  9.4 / 11.6 / 18.8
    //   512 x 3584 x 3584   15.6 / 12.6 /  8.8 / 10.2 / 12.2 / 14.3 / 19.6
    //   333 x 4863 x 896    11.4 / 10.7 /  7.5 /  7.6 /  8.3 /  9.1 / 11.7
    //   300 x 3584 x 18944  66.5 / 43.0 / 33.2 / 38.3 / 41.2 / 45.5 / 57.2
    //   64 x 18944 x 3584   19.7 / 15.1 / 13.4 / 15.5 / 16.1 / 15.7 / 19.3
    //   200 x 3584 x 3584    -   / 12.0 /  8.0 /  6.7 /  7.0 /  7.7 / 10.0
    //   124 x 3584 x 18944  72.1 / 45.6 / 34.4 / 25.6 / 19.8 / 24.1 / 31.5
    //   64 x 3584 x 18944    -   / 43.5 / 36.0 / 26.4 / 20.1 / 17.6 / 19.2
    //   64 x 3584 x 3584    15.5 / 10.7 /  7.7 /  5.9 /  4.9 /  4.7 /  5.0
    //   32 x 3584 x 3584    15.5 / 10.2 /  7.1 /  5.5 /  4.9 /  4.6 /  4.0
    //   32 x 18944 x 3584   19.5 / 14.4 / 12.3 / 13.3 / 12.7 / 11.9 / 13.8
    //   20 x 152064 x 896   23.8 / 29.9 / 20.5 / 34.0 / 19.5 / 21.5 / 30.6
    const auto count = [&](int bm, int bn) { return mx4_tile_count(M, N, bm, bn); };
    const auto kernel = [&] {
        if (M > 64 && count(128, 256) > 140)
            return Mx4Kernel::tile128x256;
        if (M > 64 && count(128, 128) >= 128)
            return Mx4Kernel::tile128x128;
        if (M > 32 && count(64, 128) >= 128)
            return Mx4Kernel::tile64x128;
        if (M > 32 && count(64, 64) >= 128)
            return Mx4Kernel::tile64x64;
        if (count(32, 64) >= 128 && (M > 32 || count(32, 32) > 1024))
            return Mx4Kernel::tile32x64;
        if (count(32, 32) >= 128)
            return Mx4Kernel::tile32x32;
        return Mx4Kernel::tile16x32;
    };
    return Mx4Shape{false, kernel()};
}

}  // namespace q4
