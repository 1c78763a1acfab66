// q4_moe_plan.hpp -- which launches the router and the expert layer take for a
// shape (host).  See q4_moe.hip for the kernels.
#pragma once

namespace q4 {

constexpr int kPart = 256;  // k of a part

// Parts of the logits in memory: all of K's, or one (the sum) from 2048 tiles
// of 16 experts by 16 rows on, where a wave a tile fills the card twice.  Router
// in us, in parts / by rows: 4096 rows x 64 experts x 2048 (1024 tiles) 43.6 /
// 50.6; 2048 x 128 x 3584 (1024) 60.7 / 72.9; 6000 x 64 x 3584 (1500) 88.8 / 109;
// 8192 x 64 x 2048 (2048) 79.9 / 79.8; 4096 x 128 x 3584 (2048) 111 / 112; 2048 x
// 512 x 1024 (4096) 168 / 164; 16384 x 128 x 2048 (8192) 278 / 250.
inline int logit_parts(int M, int E, int K)
{
    const long long tiles = (long long)((M + 15) / 16) * ((E + 15) / 16);
    return tiles >= 2048 ? 1 : (K + kPart - 1) / kPart;
}

// Whether the form that keeps a row's whole sum in a wave takes the logits.
inline bool moe_by_rows(int M, int E, int K) { return logit_parts(M, E, K) == 1 && K > kPart; }

// Whether the gate/up kernel chooses the experts itself, so that the layer is
// four launches instead of five: each of its workgroups then reads all logits'
// parts (M E parts numbers), ranks them (M E E compares) before its products
// begin, and the first writes the choice for the down kernel.  The launch costs
// about 2 us, so it pays for few numbers and few compares a thread.  Layer in
// us, within gate/up / as a launch of its own (8 or 4 or 2 choices a row):
//   experts of   896 x 512    2048 x 1024  3584 x 1792
//   1 x 64       17.9 / 19.4  21.5 / 23.7  35.6 / 38.2
//   1 x 128      19.7 / 20.6  22.7 / 24.6  37.2 / 39.1
//   16 x 8       23.1 / 24.6  25.5 / 28.3  50.2 / 51.7
//   32 x 8       27.7 / 27.9  30.4 / 32.2  55.5 / 56.5
//   4 x 64       22.4 / 22.3  36.8 / 37.6  80.0 / 76.3
//   16 x 16      25.3 / 26.8  40.2 / 41.7  64.4 / 64.0
//   8 x 36       21.8 / 19.8  28.2 / 29.1
//   32 x 12      28.1 / 25.9  40.1 / 40.8
//   16 x 32      24.9 / 24.0  45.8 / 41.1  93.5 / 81.7
//   64 x 4       33.2 / 27.2  43.4 / 44.9  63.2 / 66.5
//   64 x 8       34.6 / 27.4  41.3 / 41.8  73.5 / 71.4
//   64 x 16      40.4 / 32.3  61.0 / 54.8   122 / 106
//   256 x 8      78.7 / 44.8  92.9 / 74.8   185 / 160
//   1000 x 4      227 / 87     181 / 144    339 / 279
inline bool moe_fused(int M, int E, int K)
{
    return M <= 32 && M * E <= 256 && M * E * logit_parts(M, E, K) <= 2048 && M * E * E <= 16384;
}

}  // namespace q4
