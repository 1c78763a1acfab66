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
    // again: us fused / apart at 3584 x 3584, 1 / 2 / 4 / 8 rows 5.0 / 5.4 / 6.4 /
    // 8.3 against 6.7; 896 x 896, 1 / 8 / 16 rows 3.2 / 3.7 / 4.5 against 4.7; 3584 x
    // 18944 at one row 16.0 against 14.2.
    if (M <= 16) {
        Mx4Shape s{dense && M * K <= 14336, Mx4Kernel::relay};
        // A wave a tile of 16 columns, where every wave has one.  Fused, us relay /
        // wide: 18944 x 3584 at 1 / 4 rows 10.8 / 10.6, 14.7 / 13.0; 152064 x 896 26.0 /
        // 14.6; 3584 x 3584 5.0 / 5.5; a run of steps that holds all of K leaves the
        // relay one wave: 4864 x 896 3.7 / 3.4.  Packed rows, which the relay loads
        // beside W: 18944 x 3584 9.6 / 11.1, 32768 x 3584 13.9 / 13.4, 65536 x 3584 24.6 /
        // 23.8; 4864 x 896 2.9 / 3.3, 16384 x 896 4.3 / 4.0, 152064 x 896 22.4 / 14.6.
        const bool few_steps = mx4_steps(K) <= 8;
        const bool many = s.fused ? N >= 16384 || few_steps : N >= 32768 || (N >= 16384 && few_steps);
        if (many && mx4_few_lds(M, K) <= 60 * 1024)
            s.kernel = Mx4Kernel::wide;
        return s;
    }
    // A workgroup's chain of steps takes its time however small its tile, and what
    // passes through L2 grows as tiles shrink: the smallest tile that gives every
    // compute unit one workgroup at most, the largest where none does; rows are not
    // mostly padding.  Measured (us on packed rows, 128 x 256 / 128 x 128 / 64 x 128 /
    // 64 x 64 / 32 x 64 / 32 x 32 / 16 x 32; y bfloat16):
    //   512 x 18944 x 3584  34.2 / 39.8 / 39.1 / 47.3 / 60.3 / 67.0 / 98.4
    //   200 x 18944 x 3584  19.9 / 26.4 / 22.5 / 22.9 / 28.2 / 33.9 / 44.4
    //   512 x 8192 x 3584   18.3 / 15.9 / 18.0 / 21.6 / 27.2 / 30.8 / 43.9
    //   1024 x 3584 x 3584  15.6 / 14.7 / 16.5 / 20.0 / 23.3 / 26.6 / 37.1
    //   124 x 18944 x 3584  20.2 / 16.2 / 19.4 / 18.3 / 20.2 / 22.9 / 30.3
    //   4000 x 896 x 896    11.0 /  8.1 /  7.5 /  9.1 /  9.2 / 11.4 / 18.9
    //   512 x 4096 x 3584   15.5 / 13.2 /  9.7 / 11.6 / 13.7 / 16.4 / 21.9
    //   333 x 4863 x 896    10.9 / 10.5 /  7.2 /  7.3 /  8.0 /  8.8 / 11.5
    //   300 x 3584 x 18944  66.3 / 42.5 / 32.9 / 30.4 / 40.8 / 44.6 / 57.1
    //   64 x 18944 x 3584   19.6 / 14.6 / 12.9 / 15.0 / 15.4 / 15.2 / 18.8
    //   100 x 8192 x 3584   18.6 / 13.2 / 10.0 /  8.4 /  9.3 / 10.3 / 14.8
    //   256 x 4096 x 8192   35.4 / 22.3 / 16.6 / 12.9 / 16.0 / 18.3 / 26.1
    //   124 x 3584 x 18944  71.6 / 45.5 / 34.3 / 25.0 / 19.5 / 23.5 / 30.9
    //   40 x 8192 x 8192    34.1 / 20.9 / 17.5 / 13.1 / 11.3 / 12.4 / 14.6
    //   64 x 4096 x 8192    33.3 / 20.7 / 17.4 / 12.5 / 10.0 /  8.9 /  9.7
    //   64 x 3584 x 3584    15.3 / 10.6 /  7.5 /  5.7 /  4.7 /  4.5 /  4.9
    //   100 x 1024 x 8192   27.3 / 19.0 / 11.7 /  8.7 /  6.8 /  6.7 /  5.4
    //   32 x 3584 x 3584    15.3 / 10.2 /  7.0 /  5.5 /  4.7 /  4.5 /  3.9
    //   32 x 16384 x 3584   18.9 / 12.9 / 11.3 /  9.1 /  8.9 /  9.5 / 11.2
    //   32 x 18944 x 3584   19.5 / 14.1 / 11.7 / 12.9 / 12.3 / 11.4 / 13.0
    //   20 x 152064 x 896   23.4 / 29.0 / 19.9 / 21.7 / 19.0 / 20.8 / 30.0
    const struct {
        Mx4Kernel kernel;
        int bm, bn;
    } tiles[] = {{Mx4Kernel::tile16x32, 16, 32},     {Mx4Kernel::tile32x32, 32, 32},   {Mx4Kernel::tile32x64, 32, 64},
                 {Mx4Kernel::tile64x64, 64, 64},     {Mx4Kernel::tile64x128, 64, 128}, {Mx4Kernel::tile128x128, 128, 128},
                 {Mx4Kernel::tile128x256, 128, 256}};
    for (const auto &t : tiles)
        if (2 * M > t.bm && mx4_tile_count(M, N, t.bm, t.bn) <= kMx4Units)
            return Mx4Shape{false, t.kernel};
    const auto largest = M > 64                                 ? Mx4Kernel::tile128x256
                         : M > 32                               ? Mx4Kernel::tile64x128
                         : mx4_tile_count(M, N, 32, 32) >= 1024 ? Mx4Kernel::tile32x64
                                                                : Mx4Kernel::tile32x32;
    return Mx4Shape{false, largest};
}

}  // namespace q4
