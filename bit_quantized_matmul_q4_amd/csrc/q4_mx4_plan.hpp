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
        // beside W: 18944 x 3584 9.4 / 10.9, 32768 x 3584 13.5 / 13.1, 65536 x 3584 22.8 /
        // 22.7; 4864 x 896 2.9 / 3.3, 16384 x 896 4.3 / 4.0, 152064 x 896 22.4 / 14.6.
        const bool few_steps = mx4_steps(K) <= 8;
        const bool many = s.fused ? N >= 16384 || few_steps : N >= 32768 || (N >= 16384 && few_steps);
        if (many && mx4_few_lds(M, K) <= 60 * 1024)
            s.kernel = Mx4Kernel::wide;
        return s;
    }
    // A workgroup's chain of steps takes its time however small its tile, and what
    // passes through L2 grows as tiles shrink: the smallest tile that gives every
    // compute unit one workgroup at most; where none does, the largest of whose
    // rows more than half are there, except that up to 32 rows take 32 x 32 while
    // that is three workgroups a compute unit or fewer.  Measured (us on packed rows,
    // 128 x 256 / 128 x 128 / 64 x 128 / 64 x 64 / 32 x 64 / 32 x 32 / 16 x 32; y bfloat16;
    // replays of 24 captured calls or more over up to 24 sets of operands, 700 MB where
    // they reach it, so that W comes from memory; the seven in turn, median of 9; two
    // runs differ by up to 5%; the rule is within 9% of the best of each line):
    //   512 x 18944 x 3584  31.5 / 40.5 / 38.9 / 47.3 / 60.1 / 66.2 / 98.2
    //   200 x 18944 x 3584  19.1 / 26.4 / 22.4 / 22.7 / 28.2 / 33.8 / 44.1
    //   512 x 8192 x 3584   18.4 / 15.4 / 18.0 / 21.5 / 27.1 / 30.9 / 43.7
    //   1024 x 3584 x 3584  17.0 / 14.7 / 16.9 / 20.2 / 24.0 / 27.1 / 38.2
    //   124 x 18944 x 3584  19.7 / 16.1 / 19.1 / 18.3 / 19.9 / 22.7 / 30.1
    //   100 x 65536 x 3584  28.3 / 36.2 / 37.5 / 43.0 / 53.8 / 63.0 / 85.1
    //   100 x 32768 x 3584  21.2 / 19.4 / 21.0 / 23.5 / 28.7 / 33.6 / 44.9
    //   4000 x 896 x 896    10.9 /  8.0 /  7.5 /  9.0 /  9.1 / 11.1 / 18.2
    //   512 x 4096 x 3584   16.6 / 13.1 /  9.9 / 11.7 / 14.9 / 17.6 / 23.6
    //   333 x 4863 x 896    11.1 / 10.5 /  7.2 /  7.3 /  8.0 /  8.7 / 11.5
    //   300 x 3584 x 18944  66.1 / 42.9 / 33.1 / 30.8 / 40.6 / 44.7 / 56.9
    //   64 x 18944 x 3584   18.8 / 14.1 / 12.6 / 15.0 / 15.1 / 15.0 / 18.6
    //   64 x 65536 x 3584   29.4 / 33.1 / 29.1 / 31.4 / 36.8 / 42.2 / 54.4
    //   40 x 100000 x 3584  42.0 / 52.3 / 45.5 / 45.4 / 51.2 / 56.4 / 67.4
    //   100 x 8192 x 3584   18.5 / 13.4 / 10.1 /  8.2 /  9.4 / 10.4 / 15.0
    //   256 x 4096 x 8192   35.3 / 22.7 / 16.8 / 12.9 / 16.3 / 18.7 / 26.6
    //   124 x 3584 x 18944  71.4 / 46.1 / 34.4 / 24.9 / 19.3 / 23.5 / 30.7
    //   40 x 8192 x 8192    33.4 / 20.5 / 17.2 / 12.7 / 11.2 / 12.3 / 14.5
    //   64 x 4096 x 8192    33.0 / 20.6 / 17.3 / 12.5 / 10.1 /  9.0 /  9.8
    //   64 x 3584 x 3584    15.2 / 10.5 /  7.5 /  5.7 /  4.7 /  4.5 /  4.9
    //   100 x 1024 x 8192   27.1 / 19.0 / 11.8 /  8.8 /  7.0 /  6.7 /  5.4
    //   32 x 3584 x 3584    15.3 / 10.2 /  6.9 /  5.4 /  4.7 /  4.5 /  3.8
    //   32 x 16384 x 3584   18.3 / 12.5 / 10.8 /  8.8 /  8.5 /  9.1 / 10.9
    //   32 x 18944 x 3584   18.6 / 13.1 / 11.3 / 12.7 / 12.1 / 11.2 / 12.9
    //   32 x 24576 x 3584   19.2 / 14.4 / 12.7 / 13.8 / 13.2 / 12.6 / 15.4
    //   20 x 24576 x 896     9.5 /  6.9 /  5.6 /  5.8 /  5.5 /  5.3 /  7.1
    //   32 x 25600 x 3584   19.4 / 14.7 / 12.9 / 14.0 / 13.5 / 14.2 / 16.4
    //   20 x 25600 x 896     9.6 /  7.1 /  5.8 /  5.9 /  5.6 /  5.8 /  7.9
    //   20 x 25600 x 8192   36.2 / 24.9 / 22.2 / 24.3 / 23.4 / 25.7 / 29.6
    //   32 x 32760 x 3584   20.3 / 16.5 / 14.8 / 15.5 / 14.8 / 15.7 / 20.0
    //   20 x 152064 x 896   23.7 / 28.8 / 20.0 / 21.7 / 19.0 / 21.0 / 30.3
    const struct {
        Mx4Kernel kernel;
        int bm, bn;
    } tiles[] = {{Mx4Kernel::tile16x32, 16, 32},     {Mx4Kernel::tile32x32, 32, 32},   {Mx4Kernel::tile32x64, 32, 64},
                 {Mx4Kernel::tile64x64, 64, 64},     {Mx4Kernel::tile64x128, 64, 128}, {Mx4Kernel::tile128x128, 128, 128},
                 {Mx4Kernel::tile128x256, 128, 256}};
    for (const auto &t : tiles)
        if (2 * M > t.bm && mx4_tile_count(M, N, t.bm, t.bn) <= kMx4Units)
            return Mx4Shape{false, t.kernel};
    const auto largest = M > 64                                         ? Mx4Kernel::tile128x256
                         : M > 32                                       ? Mx4Kernel::tile64x128
                         : mx4_tile_count(M, N, 32, 32) > 3 * kMx4Units ? Mx4Kernel::tile32x64
                                                                        : Mx4Kernel::tile32x32;
    return Mx4Shape{false, largest};
}

}  // namespace q4
