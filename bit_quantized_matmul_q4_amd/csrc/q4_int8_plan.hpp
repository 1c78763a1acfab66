// q4_int8_plan.hpp -- which kernel of the 8-bit product a shape takes (host),
// and the size of its packed rows.  See q4_int8.hip for the kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace q4 {

// k64 tiles of a packed row tile (K padded to 128)
__host__ __device__ inline int int8_tiles(int K) { return 2 * ((K + 127) / 128); }

constexpr int kUnits = 256;  // compute units

// The tile and the split of K for a shape.
struct Int8Shape {
    bool decode, gemv;
    int bm, bn, split;
};

inline Int8Shape int8_shape(bool dense, int M, int N, int K)
{
    // quantizing within the product saves a launch while that is less work than
    // the launch's 2 us: 3584 x 3584 at 1 / 2 / 4 / 8 rows 5.1 / 5.7 / 6.6 / 7.6
    // against 7.2 / 7.3 / 7.8 / 7.9 us, at 12 rows 10.4 against 7.9; 18944 x
    // 3584 (more than two tiles a compute unit, each quantizing again) at one
    // row 17.0 against 14.8
    // One column tile a workgroup reads x again for each: from 17 rows on, and
    // more than 24576 columns, a 64 x 64 tile is faster (its time / the tile's at
    // 17, 32 and 64 rows, K = 3584: 3584 columns 8.4 / 11.9, 8.5 / 12.1, 10.3 /
    // 13.4; 18944 16.9 / 22.0, 17.1 / 22.2, 22.9 / 24.3; 22000 18.0 / 21.4, 18.5
    // / 22.1, 25.3 / 27.0; 26000 25.5 / 23.9, 26.0 / 23.7, 37.1 / 28.0; 152064
    // 125 / 105, 140 / 119, 189 / 125; 200 columns 7.9 / 10.2, 8.2 / 10.6, 9.6 /
    // 10.7; 3584 columns over K = 18944 19.5 / 22.4, 19.7 / 22.7, 25.9 / 25.0).
    // At 16 rows: 22000 17.0 / 20.8, 60000 48.2 / 50.3, 152064 116 / 110.
    Int8Shape s{dense && M <= 4 && M * int8_tiles(K) * 64 <= 20 * 1024 && N <= 8192,
                M <= 16 || (M <= 64 && N <= 24576), 0, 0, 1};
    if (s.decode || s.gemv)
        return s;
    // The largest tile that still fills the card, and K split while half the
    // workgroups that fit at once are missing.  Measured (us, 256 x 256 / 128 x
    // 128 / 128 x 64 / 64 x 64, the others' splits as here): 4096 x 3584 x 18944
    // (224 tiles of 256) 292 / 452 / - / -; 2048 x 3584 x 3584 (448 tiles of 128)
    // - / 42.6 / 51.9 / 62.3; 333 x 18944 x 3584 (444) - / 38.3 / 43.5 / 48.3;
    // 1024 x 3584 x 3584 (224) - / 33.3 / 28.1 / 34.8; 512 x 3584 x 3584 (112) -
    // / 25.9 / 24.5 / 21.9; 124 x 3584 x 18944 (28) - / 34.1 / 33.0 / 30.5.  Tiles
    // taller than the rows multiply padding: 48 x 152064 x 3584 - / 127 / - / 127,
    // 48 x 152064 x 896 - / 47.1 / - / 42.8, 48 x 32000 x 3584 - / - / 32.8 / 30.6;
    // 65 x 152064 x 3584 153 / 130 / - / 144, 128 x 152064 x 3584 166 / 152 / - / 179,
    // 128 x 60000 x 896 25.2 / 21.0 / - / 24.2; but 129 x 152064 x 3584 161 / 171.
    const auto count = [&](int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
    int at_once;
    if (M > 128 && count(256, 256) >= 200) {
        s.bm = s.bn = 256;
        at_once = kUnits;
    } else if (M > 64 && count(128, 128) >= 400) {
        s.bm = s.bn = 128;
        at_once = 2 * kUnits;
    } else if (M > 64 && count(128, 128) >= 200) {
        s.bm = 128;
        s.bn = 64;
        at_once = 2 * kUnits;
    } else {
        s.bm = s.bn = 64;
        at_once = 3 * kUnits;
    }
    const long long wgs = count(s.bm, s.bn);
    const int steps = int8_tiles(K) / 2;
    while (2 * wgs * s.split <= at_once && steps / (2 * s.split) >= 4)
        s.split *= 2;
    return s;
}

// Rows a workgroup of the quantizer (16 were slower everywhere: 4096 x 3584, from
// the last-level cache, in 23 us against 12 with four; one against four at 1024
// rows 31.2 against 32.5 us with the product, at 4096 rows 306 against 299).
inline int quant_rows(int rows) { return rows >= 2048 ? 4 : 1; }

}  // namespace q4
