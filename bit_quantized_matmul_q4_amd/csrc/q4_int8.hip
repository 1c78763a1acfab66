// q4_int8.hip -- the matrix product in 8-bit integers for gfx950 (MI355X):
//
//     y[m][n] = (sum_k qx[m][k] qw[n][k]) sx[m] sw[n]
//
// with one binary32 scale for each row of x (token) and each row of W
// (channel).  The sum is a 32-bit integer and exact, so a row's bits depend
// on the row alone: not on M, the kernel, the tile or the split of K.
//
// Row quantizer: a = max |x[m]|; s = a / 127 rounded once to binary32;
// q = clamp(round_half_even(x / s), -127, 127) on the exact quotient.  A row
// of zeros has s = 0 and codes 0; a row that holds an infinity or NaN has
// s = NaN and codes 0, so its outputs are NaN and no other row's are.
//
// Packed layout of both operands (q4.h): tiles of 16 rows by 64 k in the
// order [ceil(rows / 16)][2 ceil(K / 128)], 1024 bytes each; lane l = 16 g +
// c of a wave owns bytes 16 l .. 16 l + 15: row 16 t + c, k = 64 q + 16 g ..
// + 15.  That is the operand order of v_mfma_i32_16x16x64_i8, so a wave's
// loads from memory and from LDS are contiguous and need no swizzle.
// Padding rows and padding k are zero.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "q4_int8_plan.hpp"
#include "q4_launch.hpp"

namespace q4 {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------- quantizer
// Element types: 0 binary16, 1 bfloat16, 2 binary32.
template <int KIND>
using Elem = std::conditional_t<KIND == 2, uint32_t, uint16_t>;

template <int KIND>
__device__ __forceinline__ float elem_value(uint32_t bits)
{
    if constexpr (KIND == 2)
        return __builtin_bit_cast(float, bits);
    else if constexpr (KIND == 1)
        return __builtin_bit_cast(float, bits << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// Largest |x| as ordered bits: the sign dropped, infinities and NaN above
// every finite value.
template <int KIND>
constexpr uint32_t kAbsMask = KIND == 2 ? 0x7FFFFFFFu : 0x7FFFu;
template <int KIND>
constexpr uint32_t kInfBits = KIND == 2 ? 0x7F800000u : KIND == 1 ? 0x7F80u : 0x7C00u;

// What a row's codes are made with: lift (a power of two that keeps the
// quotient's operands normal), the lifted scale and its approximate inverse.
struct RowScale {
    float scale, lift, s, inv;
};

template <int KIND>
__device__ __forceinline__ RowScale row_scale(uint32_t top)
{
    RowScale r;
    if (top >= kInfBits<KIND>) {
        r.scale = __builtin_nanf("");
        r.lift = r.s = r.inv = 0.f;
        return r;
    }
    const float a = elem_value<KIND>(top);
    r.scale = a / 127.f;
    r.lift = a < 0x1p-90f ? 0x1p100f : 1.f;
    r.s = r.scale * r.lift;  // exact
    r.inv = r.s > 0.f ? 1.f / r.s : 0.f;
    return r;
}

// round_half_even(x / s), exactly: an estimate from the inverse (off by one
// at most, and only next to a border), put right by the remainder x - r s,
// which one fma gives without rounding (it is a multiple of ulp(s) / 2 and
// at most about s).
__device__ __forceinline__ int row_code(float x, const RowScale &r)
{
    if (!(r.s > 0.f))
        return 0;
    x *= r.lift;
    float q = __builtin_rintf(x * r.inv);
    const float e = __builtin_fmaf(-q, r.s, x);
    const float e2 = 2.f * __builtin_fabsf(e);
    const bool odd = ((int)q & 1) != 0;
    if (e2 > r.s || (e2 == r.s && odd))
        q += __builtin_copysignf(1.f, e);
    return (int)__builtin_fminf(__builtin_fmaxf(q, -127.f), 127.f);
}

// 16 values of a row: their largest magnitude's bits, and their codes.
template <int KIND, int VECS>
__device__ __forceinline__ uint32_t top_of(const u32x4 (&v)[VECS])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            top = max(top, v[i][j] & kAbsMask<KIND>);
            if constexpr (KIND != 2)
                top = max(top, (v[i][j] >> 16) & kAbsMask<KIND>);
        }
    return top;
}
template <int KIND, int VECS>
__device__ __forceinline__ float value_of(const u32x4 (&v)[VECS], int e)
{
    uint32_t bits;
    if constexpr (KIND == 2)
        bits = v[e / 4][e % 4];
    else
        bits = (v[e / 8][(e / 2) % 4] >> (16 * (e & 1))) & 0xFFFFu;
    return elem_value<KIND>(bits);
}

// The codes by the inverse: one fma rounds x / s (within 127 2^-23 of the
// quotient) to a whole number in the low bits of 1.5 2^23 + q, and a second
// one gives what is left, at most 1/2.  Where all 16 are further from a border
// than the inverse can be off, the codes are exact; else (4 in 100000 values
// of a smooth distribution), and where the scale is so small that it was
// lifted, they are taken one by one.
template <int KIND, int VECS>
__device__ __forceinline__ u32x4 codes_of(const u32x4 (&v)[VECS], const RowScale &rs)
{
    constexpr float magic = 0x1.8p23f;
    u32x4 out;
    float left = rs.lift == 1.f ? 0.f : 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t u[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const float x = value_of<KIND>(v, 4 * j + b);
            const float t = __builtin_fmaf(x, rs.inv, magic);
            left = __builtin_fmaxf(left, __builtin_fabsf(__builtin_fmaf(x, rs.inv, -(t - magic))));
            u[b] = __builtin_bit_cast(uint32_t, t);
        }
        const uint32_t lo = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u);  // bytes 0 of u[0] and u[1]
        const uint32_t hi = __builtin_amdgcn_perm(u[3], u[2], 0x04000c0cu);
        out[j] = lo | hi;
    }
    if (!(left < 0.49996f)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t word = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                word |= ((uint32_t)row_code(value_of<KIND>(v, 4 * j + b), rs) & 0xFFu) << (8 * b);
            out[j] = word;
        }
    }
    return out;
}

// One workgroup quantizes RW rows (a divisor of 16); a wave's 64 lanes are RW
// rows by 64 / RW pieces of 16 k.  One row a workgroup spreads few rows over
// the card, several make the pieces of a packed tile that a wave writes lie
// together.  Two passes over the row: the largest |x|, then the codes; the
// second takes the first HELD pieces of each lane from registers (a row of
// 32768 with one row a workgroup) and the rest from the L2.
// PACKED: the packed layout (padding written), else codes [rows][K].
// grid = row groups (PACKED: of the padded rows, so that padding rows are
// written too).  Bound by memory latency for few rows (4 us at 8 x 3584, 8 at
// 124 x 18944), by memory for many: 4096 x 3584 in 15 us, 2.9 TB/s, from rows
// that no cache holds.
constexpr int kQuantThreads = 512;

template <int KIND, int RW, bool PACKED>
__global__ __launch_bounds__(kQuantThreads) void q4_int8_quantize_kernel(const void *__restrict__ x_,
                                                                       int8_t *__restrict__ codes,
                                                                       float *__restrict__ scales, int rows, int K)
{
    typedef Elem<KIND> E;
    constexpr int PIECES = 64 / RW;                     // pieces of 16 k a wave step covers
    constexpr int STEP = PIECES * (kQuantThreads / 64);  // and the workgroup's
    constexpr int HELD = KIND == 2 ? 2 : 4;
    constexpr int VECS = (int)sizeof(E);  // 16-byte vectors a piece
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int c = lane % RW, p0 = wave * PIECES + lane / RW;
    const int row = blockIdx.x * RW + c;
    const bool live = row < rows;
    const int pieces = K / 16;
    const E *x = (const E *)x_ + (size_t)(live ? row : 0) * K;

    u32x4 held[HELD][VECS];
    uint32_t top = 0;
    auto load = [&](int p, u32x4 (&v)[VECS]) {
        const u32x4 *src = (const u32x4 *)(x + 16 * (size_t)p);
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            v[i] = src[i];
    };
    if (live) {
#pragma unroll
        for (int h = 0; h < HELD; ++h)
            if (p0 + h * STEP < pieces)
                load(p0 + h * STEP, held[h]);
#pragma unroll
        for (int h = 0; h < HELD; ++h)
            if (p0 + h * STEP < pieces)
                top = max(top, top_of<KIND>(held[h]));
        for (int p = p0 + HELD * STEP; p < pieces; p += STEP) {
            u32x4 v[VECS];
            load(p, v);
            top = max(top, top_of<KIND>(v));
        }
    }
    // over the lanes and waves of the same row
    __shared__ uint32_t tops[kQuantThreads / 64][RW];
#pragma unroll
    for (int d = RW; d < 64; d *= 2)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (lane < RW)
        tops[wave][lane] = top;
    __syncthreads();
    top = 0;
#pragma unroll
    for (int w = 0; w < kQuantThreads / 64; ++w)
        top = max(top, tops[w][c]);
    const RowScale rs = row_scale<KIND>(top);
    if (live && threadIdx.x < RW)
        scales[row] = rs.scale;

    const int tiles = int8_tiles(K);
    const int all = PACKED ? 4 * tiles : pieces;
    auto store = [&](int p, u32x4 v) {
        if constexpr (PACKED) {
            const size_t tile = (size_t)(row >> 4) * tiles + (p >> 2);
            *(u32x4 *)(codes + tile * 1024 + (p & 3) * 256 + (row & 15) * 16) = v;
        } else if (live) {
            *(u32x4 *)(codes + (size_t)row * K + 16 * (size_t)p) = v;
        }
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
        const int p = p0 + h * STEP;
        if (p < all)
            store(p, live && p < pieces ? codes_of<KIND>(held[h], rs) : (u32x4){0, 0, 0, 0});
    }
    for (int p = p0 + HELD * STEP; p < all; p += STEP) {
        u32x4 v[VECS];
        if (live && p < pieces) {
            load(p, v);
            store(p, codes_of<KIND>(v, rs));
        } else {
            store(p, (u32x4){0, 0, 0, 0});
        }
    }
}

// Canonical codes [rows][K] -> packed, 16 bytes a thread.
__global__ __launch_bounds__(256) void q4_int8_pack_kernel(const int8_t *__restrict__ codes,
                                                           int8_t *__restrict__ packed, int rows, int K, size_t items)
{
    const int tiles = int8_tiles(K);
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (size_t)gridDim.x * 256) {
        const int lane = (int)(i & 63);
        const size_t tile = i >> 6;
        const size_t row = tile / tiles * 16 + (lane & 15);
        const int k = (int)(tile % tiles) * 64 + 16 * (lane >> 4);
        u32x4 v = {0, 0, 0, 0};
        if (row < (size_t)rows && k < K)
            v = *(const u32x4 *)(codes + row * K + k);
        *(u32x4 *)(packed + i * 16) = v;
    }
}

// --------------------------------------------------------------- outputs
// Output types: 0 binary16, 1 bfloat16, 2 binary32.
// A scale as mantissa in [0.5, 1) and exponent: the output's value is
// float(sum) times both mantissas (three roundings), then one ldexp by both
// exponents, so that no product on the way overflows or underflows where the
// value does not (a huge activation scale against a tiny weight scale).
struct Scale {
    float m;
    int e;
};
__device__ __forceinline__ Scale split_scale(float s)
{
    return Scale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}
__device__ __forceinline__ float scaled(int sum, Scale sx, Scale sw)
{
    return __builtin_ldexpf((float)sum * sx.m * sw.m, sx.e + sw.e);
}

__device__ __forceinline__ uint16_t bf16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint16_t f16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Four consecutive outputs n .. n + 3 of row m (those below N), as one store
// where `vec` says that rows start aligned.
template <int YK>
__device__ __forceinline__ void store4(void *y, size_t at, int left, bool vec, f32x4 v)
{
    if constexpr (YK == 2) {
        float *p = (float *)y + at;
        if (vec && left >= 4) {
            *(f32x4 *)p = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left)
                    p[i] = v[i];
        }
    } else {
        uint16_t *p = (uint16_t *)y + at;
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = YK == 1 ? bf16_bits(v[i]) : f16_bits(v[i]);
        if (vec && left >= 4) {
            *(uint2 *)p = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left)
                    p[i] = h[i];
        }
    }
}

__device__ __forceinline__ f32x4 scaled4(i32x4 a, Scale sx, const Scale (&sw)[4])
{
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = scaled(a[i], sx, sw[i]);
    return v;
}

// --------------------------------------------------------------- few rows
// Up to 16 RT rows of x: bound by the bytes of W.  A workgroup owns one tile
// of 16 columns; its waves take the tile's k64 steps in turn, U at a time,
// and their integer sums meet in LDS.  18944 x 3584 at 8 rows: 14.7 to 15.4 us, 4.4
// to 4.6 TB/s, with weights from memory (a plain read of 1 GiB: 6.3), 11.8 us with
// weights that the last-level cache holds.
template <int RT, int YK>
__global__ __launch_bounds__(512) void q4_int8_gemv_kernel(const int8_t *__restrict__ xq, const float *__restrict__ sx,
                                                           const int8_t *__restrict__ wq, const float *__restrict__ sw,
                                                           void *__restrict__ y, int M, int N, int K, int vec)
{
    constexpr int W = 8;
    constexpr int U = RT >= 4 ? 2 : 4;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int tiles = int8_tiles(K);
    const int8_t *w = wq + (size_t)blockIdx.x * tiles * 1024 + lane * 16;
    const int8_t *x = xq + lane * 16;
    const size_t xrow = (size_t)tiles * 1024;
    const int rows = (M + 15) / 16;  // row tiles (one past the end: the last, its outputs are not stored)
    i32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        acc[r] = (i32x4){0, 0, 0, 0};
    for (int q0 = wave; q0 < tiles; q0 += W * U) {
        i32x4 a[U], b[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = q0 + u * W;
            if (q < tiles) {
                a[u] = *(const i32x4 *)(w + (size_t)q * 1024);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    b[u][r] = *(const i32x4 *)(x + min(r, rows - 1) * xrow + (size_t)q * 1024);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q0 + u * W < tiles) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], b[u][r], acc[r], 0, 0, 0);
            }
    }
    __shared__ i32x4 part[W][RT][64];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        part[wave][r][lane] = acc[r];
    __syncthreads();
    for (int r = wave; r < RT; r += W) {
        i32x4 s = part[0][r][lane];
#pragma unroll
        for (int j = 1; j < W; ++j)
            s += part[j][r][lane];
        const int m = 16 * r + (lane & 15), n = 16 * blockIdx.x + 4 * (lane >> 4);
        if (m < M && n < N) {
            Scale ws[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ws[i] = split_scale(n + i < N ? sw[n + i] : 0.f);
            store4<YK>(y, (size_t)m * N + n, N - n, vec, scaled4(s, split_scale(sx[m]), ws));
        }
    }
}

// ------------------------------------------------------- a few dense rows
// A few dense rows in one launch: a workgroup quantizes all of them into LDS (M
// K bytes) while its first weights are on their way, then multiplies its tile
// of W.  A wave takes every eighth k64 step, in chunks of eight steps, one
// chunk ahead of the products.  3584 x 3584 at one row: 5.8 us (5.1 with W in the
// last-level cache), of which the launch and two memory latencies (x, then W) are
// most.
constexpr uint32_t kNowhere = 1u << 31;  // past every tile's range: reads zero, no access
constexpr int kDecodeWaves = 8, kDecodeChunk = 8;

template <int KIND, int YK>
__global__ __launch_bounds__(64 * kDecodeWaves) void q4_int8_decode_kernel(const void *__restrict__ x_,
                                                                           const int8_t *__restrict__ wq,
                                                                           const float *__restrict__ sw,
                                                                           void *__restrict__ y, int M, int N, int K,
                                                                           int vec)
{
    constexpr int W = kDecodeWaves, U = kDecodeChunk;
    extern __shared__ __attribute__((aligned(16))) int8_t xl[];  // [k16 piece][row][16]
    __shared__ i32x4 part[W][64];
    __shared__ uint32_t tops[4];
    __shared__ float scale_of[4];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int g = lane >> 4, c = min(lane & 15, M - 1);
    const int steps = int8_tiles(K);
    const __amdgpu_buffer_rsrc_t wb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t *>(wq + (size_t)blockIdx.x * steps * 1024), (short)0, steps * 1024, 0x00020000);
    auto fetch = [&](u32x4 (&v)[U], int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + W * u + wave;
            v[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 wb, s < steps ? s * 1024 + lane * 16 : kNowhere, 0, 2));
        }
    };
    u32x4 w0[U], w1[U];
    fetch(w0, 0);

    // the rows: W / per of them at once, at least M (at most 4: see int8_shape)
    {
        typedef Elem<KIND> E;
        constexpr int HELD = 2, VECS = (int)sizeof(E);
        int per = W;
        while (W / per < M)
            per /= 2;
        const int row = wave / per, pieces = K / 16, step = 64 * per, p0 = (wave % per) * 64 + lane;
        const E *x = (const E *)x_ + (size_t)min(row, M - 1) * K;
        u32x4 held[HELD][VECS];
        uint32_t top = 0;
        auto load = [&](int p, u32x4 (&v)[VECS]) {
#pragma unroll
            for (int i = 0; i < VECS; ++i)
                v[i] = *((const u32x4 *)(x + 16 * (size_t)p) + i);
        };
        if (tid < 4)
            tops[tid] = 0;
        __syncthreads();
        if (row < M) {
#pragma unroll
            for (int h = 0; h < HELD; ++h)
                if (p0 + h * step < pieces)
                    load(p0 + h * step, held[h]);
#pragma unroll
            for (int h = 0; h < HELD; ++h)
                if (p0 + h * step < pieces)
                    top = max(top, top_of<KIND>(held[h]));
            for (int p = p0 + HELD * step; p < pieces; p += step) {
                u32x4 v[VECS];
                load(p, v);
                top = max(top, top_of<KIND>(v));
            }
#pragma unroll
            for (int d = 1; d < 64; d *= 2)
                top = max(top, (uint32_t)__shfl_xor((int)top, d));
            if (lane == 0)
                atomicMax(&tops[row], top);
        }
        __syncthreads();
        if (row < M) {
            const RowScale rs = row_scale<KIND>(tops[row]);
            if (p0 == 0)
                scale_of[row] = rs.scale;
            for (int h = 0, p = p0; p < 4 * steps; ++h, p += step) {
                u32x4 v = {0, 0, 0, 0};
                if (p < pieces) {
                    if (h >= HELD) {
                        u32x4 raw[VECS];
                        load(p, raw);
                        v = codes_of<KIND>(raw, rs);
                    } else {
                        v = codes_of<KIND>(h == 0 ? held[0] : held[1], rs);
                    }
                }
                *(u32x4 *)(xl + ((size_t)p * M + row) * 16) = v;
            }
        }
        __syncthreads();
    }

    const int8_t *xr = xl + (g * M + c) * 16;
    i32x4 acc = {0, 0, 0, 0};
    auto multiply = [&](const u32x4 (&v)[U], int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {  // (steps past the end: zero weights, the last values again)
            const int s = min(s0 + W * u + wave, steps - 1);
            const i32x4 b = *(const i32x4 *)(xr + (size_t)s * 64 * M);
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, v[u]), b, acc, 0, 0, 0);
        }
    };
    for (int s0 = 0; s0 < steps; s0 += 2 * W * U) {
        fetch(w1, s0 + W * U);
        multiply(w0, s0);
        fetch(w0, s0 + 2 * W * U);
        if (s0 + W * U < steps)
            multiply(w1, s0 + W * U);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        i32x4 s = part[0][lane];
#pragma unroll
        for (int j = 1; j < W; ++j)
            s += part[j][lane];
        const int m = lane & 15, n = 16 * blockIdx.x + 4 * g;
        if (m < M && n < N) {
            Scale ws[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ws[i] = split_scale(n + i < N ? sw[n + i] : 0.f);
            store4<YK>(y, (size_t)m * N + n, N - n, vec, scaled4(s, split_scale(scale_of[m]), ws));
        }
    }
}

// -------------------------------------------------------------- many rows
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t src, int8_t *lds, int lane_at, int at)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void *)lds, 16, lane_at, at, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// LDS-tiled: a workgroup of WM x WN waves owns BM rows by BN columns; steps of
// 128 k go from memory to LDS directly, NS stages deep.  Within a step a wave
// reads the operands of one half (64 k) from LDS while it multiplies the
// other: the barrier that frees a stage falls between the halves, when both
// halves' operands of the step are in registers, so that neither the LDS reads
// nor the loads of the next stages hold up the matrix cores.
// 4096 x 18944 x 3584 (256 x 256): 281 to 287 us, 1.94 to 1.98 Pop/s, in a captured
// replay, 292 to 298 with a tracer beside it.  Taken apart in builds of their own, of then 285
// us: the products alone, on operands that stay in registers, 208 us (the card's
// clock falls under them), with the LDS reads 237, with the loads but no reads
// 270.  With the 32 x 32 x 32 form of the instruction the whole took 17 us more,
// with four waves of 128 x 128 65 us more (copies between register files).
template <int BM, int BN, int WM, int WN, int NS, int YK>
__global__ __launch_bounds__(64 * WM *WN) void q4_int8_gemm_kernel(
    const int8_t *__restrict__ xq, const float *__restrict__ sx, const int8_t *__restrict__ wq,
    const float *__restrict__ sw, void *__restrict__ y, int *__restrict__ partial, int M, int N, int K, int steps_per,
    int vec)
{
    constexpr int WAVES = WM * WN;
    constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN;  // a wave's row tiles of x and of W
    constexpr int CHUNKS = (BM + BN) / 16 * 2;           // 1 KB pieces of a stage
    static_assert(BM / 8 % WAVES == 0 && BN / 8 % WAVES == 0, "every wave loads as many pieces of each operand");
    constexpr int PER = CHUNKS / WAVES, PER_X = BM / 8 / WAVES;
    constexpr int STAGE = CHUNKS * 1024;
    extern __shared__ __attribute__((aligned(16))) int8_t lds[];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave % WM, wn = wave / WM;
    const int tiles = int8_tiles(K);
    const int tm_all = (M + 15) / 16, tn_all = (N + 15) / 16;
    const int gm = (M + BM - 1) / BM, gn = (N + BN - 1) / BN;
    // workgroups go to the 8 dies in turn: each die takes a run of tiles, in
    // bands of four row tiles, so that few panels of x and W pass through its L2
    // at once (8192 x 4096 x 4096: 170 us with all row tiles in one band, 152
    // with four)
    int id = blockIdx.x;
    {
        const int total = gm * gn, q = total / 8, r = total % 8, die = id & 7;
        id = die * q + min(die, r) + (id >> 3);
    }
    const int group = id / (4 * gn), rows_in = min(4, gm - 4 * group), in_group = id - 4 * group * gn;
    const int bm = 4 * group + in_group % rows_in, bn = in_group / rows_in;
    const int s0 = blockIdx.y * steps_per, s1 = min(tiles / 2, s0 + steps_per);

    // the pieces this wave loads, every WAVES-th: first of x, then of W (row
    // tiles past the end: the last one, its outputs are not stored)
    const int mt = bm * (BM / 16), nt = bn * (BN / 16);
    const __amdgpu_buffer_rsrc_t xb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t *>(xq + (size_t)mt * tiles * 1024), (short)0, min(tm_all - mt, BM / 16) * tiles * 1024,
        0x00020000);
    const __amdgpu_buffer_rsrc_t wb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t *>(wq + (size_t)nt * tiles * 1024), (short)0, min(tn_all - nt, BN / 16) * tiles * 1024,
        0x00020000);
    int at[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int ch = (i < PER_X ? i : i - PER_X) * WAVES + wave;
        at[i] = min(ch / 2, i < PER_X ? tm_all - 1 - mt : tn_all - 1 - nt) * tiles * 1024 + (ch & 1) * 1024;
    }
    auto fetch = [&](int step) {  // (past the last step: the last again, so that the counts stay)
        const int stage = (step - s0) % NS, off = min(step, s1 - 1) * 2048;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            load_lds(i < PER_X ? xb : wb, lds + stage * STAGE + (i * WAVES + wave) * 1024, lane * 16, at[i] + off);
    };
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = (i32x4){0, 0, 0, 0};
    i32x4 a[2][TN], b[2][TM];
    auto read = [&](int half, int step) {
        const int8_t *p = lds + (step - s0) % NS * STAGE + lane * 16 + half * 1024;
#pragma unroll
        for (int j = 0; j < TM; ++j)
            b[half][j] = *(const i32x4 *)(p + (wm * TM + j) * 2048);
#pragma unroll
        for (int i = 0; i < TN; ++i)
            a[half][i] = *(const i32x4 *)(p + (BM / 16 + wn * TN + i) * 2048);
    };
    auto multiply = [&](int half) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[half][i], b[half][j], acc[i][j], 0, 0, 0);
    };
    if (s0 < s1) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            fetch(s0 + i);
        wait_loads<PER *(NS - 1)>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(0, s0);
        for (int s = s0; s < s1; ++s) {
            read(1, s);
            __builtin_amdgcn_sched_barrier(0);
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
            // this wave's reads of step s are done, and its pieces of step s + 1 here
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            wait_loads<PER *(NS - 2)>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            fetch(s + NS);
            if (s + 1 < s1)
                read(0, s + 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(1);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_loads<0>();  // (the loads past the end: nothing is in flight into LDS when the workgroup ends)
    }
    // lane (g, c) holds row c of a tile of x, rows 4 g .. 4 g + 3 of one of W
    const int m0 = bm * BM + wm * TM * 16 + (lane & 15), n0 = bn * BN + wn * TN * 16 + 4 * (lane >> 4);
    if (partial) {  // a split's sums as they lie: [split][tile of W][tile of x][lane]
        i32x4 *out = (i32x4 *)partial + (size_t)blockIdx.y * tn_all * tm_all * 64 + lane;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int tn = nt + wn * TN + i, tm = mt + wm * TM + j;
                if (tn < tn_all && tm < tm_all)
                    out[((size_t)tn * tm_all + tm) * 64] = acc[i][j];
            }
        return;
    }
    Scale xs[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j)
        xs[j] = split_scale(m0 + 16 * j < M ? sx[m0 + 16 * j] : 0.f);
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        const int n = n0 + 16 * i;
        Scale ws[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ws[e] = split_scale(n + e < N ? sw[n + e] : 0.f);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int m = m0 + 16 * j;
            if (m < M && n < N)
                store4<YK>(y, (size_t)m * N + n, N - n, vec, scaled4(acc[i][j], xs[j], ws));
        }
    }
}

// The splits' sums, added and scaled: a wave a tile of 16 x 16.  One memory
// latency: 3 to 5 us.
template <int YK>
__global__ __launch_bounds__(256) void q4_int8_join_kernel(const i32x4 *__restrict__ partial,
                                                           const float *__restrict__ sx, const float *__restrict__ sw,
                                                           void *__restrict__ y, int M, int N, int split, int vec)
{
    const int tm_all = (M + 15) / 16, tn_all = (N + 15) / 16, lane = threadIdx.x & 63;
    const int all = tm_all * tn_all, tile = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (tile >= all)
        return;
    const int m = tile % tm_all * 16 + (lane & 15), n = tile / tm_all * 16 + 4 * (lane >> 4);
    i32x4 s = {0, 0, 0, 0};
    for (int j0 = 0; j0 < split; j0 += 8) {
        i32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = partial[((size_t)min(j0 + j, split - 1) * all + tile) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < split)
                s += v[j];
    }
    if (m >= M || n >= N)
        return;
    Scale ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ws[i] = split_scale(n + i < N ? sw[n + i] : 0.f);
    store4<YK>(y, (size_t)m * N + n, N - n, vec, scaled4(s, split_scale(sx[m]), ws));
}

template <int KIND, int RW, bool PACKED>
void launch_rows(const void *x, int8_t *codes, float *scales, int rows, int K, hipStream_t stream)
{
    const int groups = PACKED ? (rows + 15) / 16 * 16 / RW : (rows + RW - 1) / RW;
    hipLaunchKernelGGL((q4_int8_quantize_kernel<KIND, RW, PACKED>), dim3((unsigned)groups), dim3(kQuantThreads), 0,
                       stream, x, codes, scales, rows, K);
}

template <int KIND, bool PACKED>
void launch_rows_k(const void *x, int8_t *codes, float *scales, int rows, int K, hipStream_t stream)
{
    if (quant_rows(rows) == 4)
        launch_rows<KIND, 4, PACKED>(x, codes, scales, rows, K, stream);
    else
        launch_rows<KIND, 1, PACKED>(x, codes, scales, rows, K, stream);
}

template <int RT>
void launch_gemv_rt(int yk, const int8_t *xq, const float *sx, const int8_t *wq, const float *sw, void *y, int M, int N,
                    int K, int vec, hipStream_t stream)
{
    const dim3 grid((unsigned)((N + 15) / 16)), block(512);
    if (yk == 2)
        hipLaunchKernelGGL((q4_int8_gemv_kernel<RT, 2>), grid, block, 0, stream, xq, sx, wq, sw, y, M, N, K, vec);
    else if (yk == 1)
        hipLaunchKernelGGL((q4_int8_gemv_kernel<RT, 1>), grid, block, 0, stream, xq, sx, wq, sw, y, M, N, K, vec);
    else
        hipLaunchKernelGGL((q4_int8_gemv_kernel<RT, 0>), grid, block, 0, stream, xq, sx, wq, sw, y, M, N, K, vec);
}

template <int BM, int BN, int WM, int WN, int NS, int YK>
hipError_t launch_tile_y(const int8_t *xq, const float *sx, const int8_t *wq, const float *sw, void *y, int *partial,
                         int M, int N, int K, int split, int vec, hipStream_t stream)
{
    constexpr int kLds = NS * (BM + BN) / 16 * 2 * 1024;
    if (kLds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void *)q4_int8_gemm_kernel<BM, BN, WM, WN, NS, YK>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (e != hipSuccess)
            return e;
    }
    const int steps = int8_tiles(K) / 2;
    const dim3 grid((unsigned)((M + BM - 1) / BM * ((N + BN - 1) / BN)), (unsigned)split);
    hipLaunchKernelGGL((q4_int8_gemm_kernel<BM, BN, WM, WN, NS, YK>), grid, dim3(64 * WM * WN), kLds, stream, xq, sx, wq, sw,
                       y, partial, M, N, K, (steps + split - 1) / split, vec);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NS>
hipError_t launch_tile(int yk, const int8_t *xq, const float *sx, const int8_t *wq, const float *sw, void *y,
                       int *partial, int M, int N, int K, int split, int vec, hipStream_t stream)
{
    if (yk == 2)
        return launch_tile_y<BM, BN, WM, WN, NS, 2>(xq, sx, wq, sw, y, partial, M, N, K, split, vec, stream);
    if (yk == 1)
        return launch_tile_y<BM, BN, WM, WN, NS, 1>(xq, sx, wq, sw, y, partial, M, N, K, split, vec, stream);
    return launch_tile_y<BM, BN, WM, WN, NS, 0>(xq, sx, wq, sw, y, partial, M, N, K, split, vec, stream);
}

template <int KIND, int YK>
hipError_t launch_decode_y(const void *x, const int8_t *wq, const float *sw, void *y, int M, int N, int K, int vec,
                           hipStream_t stream)
{
    hipLaunchKernelGGL((q4_int8_decode_kernel<KIND, YK>), dim3((unsigned)((N + 15) / 16)), dim3(64 * kDecodeWaves),
                       (size_t)M * int8_tiles(K) * 64, stream, x, wq, sw, y, M, N, K, vec);
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_decode(const void *x, const int8_t *wq, const float *sw, void *y, int yk, int M, int N, int K, int vec,
                         hipStream_t stream)
{
    if (yk == 2)
        return launch_decode_y<KIND, 2>(x, wq, sw, y, M, N, K, vec, stream);
    if (yk == 1)
        return launch_decode_y<KIND, 1>(x, wq, sw, y, M, N, K, vec, stream);
    return launch_decode_y<KIND, 0>(x, wq, sw, y, M, N, K, vec, stream);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t int8_packed_bytes(int rows, int K) { return (size_t)((rows + 15) / 16) * int8_tiles(K) * 1024; }

hipError_t launch_int8_quantize(const void *x, int kind, int8_t *codes, bool packed, float *scales, int rows, int K,
                                hipStream_t stream)
{
    if (packed) {
        if (kind == 2)
            launch_rows_k<2, true>(x, codes, scales, rows, K, stream);
        else if (kind == 1)
            launch_rows_k<1, true>(x, codes, scales, rows, K, stream);
        else
            launch_rows_k<0, true>(x, codes, scales, rows, K, stream);
    } else {
        if (kind == 2)
            launch_rows_k<2, false>(x, codes, scales, rows, K, stream);
        else if (kind == 1)
            launch_rows_k<1, false>(x, codes, scales, rows, K, stream);
        else
            launch_rows_k<0, false>(x, codes, scales, rows, K, stream);
    }
    return hipGetLastError();
}

hipError_t launch_int8_pack(const int8_t *codes, int8_t *packed, int rows, int K, hipStream_t stream)
{
    const size_t items = int8_packed_bytes(rows, K) / 16;
    hipLaunchKernelGGL(q4_int8_pack_kernel, dim3((unsigned)std::min<size_t>((items + 255) / 256, 1 << 16)), dim3(256), 0,
                       stream, codes, packed, rows, K, items);
    return hipGetLastError();
}

size_t int8_workspace_bytes(bool dense, int M, int N, int K)
{
    const Int8Shape sh = int8_shape(dense, M, N, K);
    size_t n = 0;
    if (dense && !sh.decode)
        n += up256(int8_packed_bytes(M, K)) + up256((size_t)M * sizeof(float));
    if (sh.split > 1)
        n += (size_t)sh.split * ((M + 15) / 16) * ((N + 15) / 16) * 1024;
    return n;
}

hipError_t launch_int8_linear(const void *x, int x_kind, const float *x_scales, const int8_t *wq, const float *w_scales,
                              void *y, int y_kind, int M, int N, int K, void *workspace, hipStream_t stream)
{
    const Int8Shape sh = int8_shape(x_kind >= 0, M, N, K);
    const int size = y_kind == 2 ? 4 : 2;
    const int vec = N % 4 == 0 && ((uintptr_t)y & (4 * size - 1)) == 0;
    if (sh.decode)
        return x_kind == 1 ? launch_decode<1>(x, wq, w_scales, y, y_kind, M, N, K, vec, stream)
                           : launch_decode<0>(x, wq, w_scales, y, y_kind, M, N, K, vec, stream);
    uint8_t *ws = (uint8_t *)workspace;
    const int8_t *xq = (const int8_t *)x;
    const float *sx = x_scales;
    if (x_kind >= 0) {
        int8_t *q = (int8_t *)ws;
        ws += up256(int8_packed_bytes(M, K));
        float *s = (float *)ws;
        ws += up256((size_t)M * sizeof(float));
        const hipError_t e = launch_int8_quantize(x, x_kind, q, true, s, M, K, stream);
        if (e != hipSuccess)
            return e;
        xq = q;
        sx = s;
    }
    if (sh.gemv) {
        const int rt = (M + 15) / 16;
        if (rt == 1)
            launch_gemv_rt<1>(y_kind, xq, sx, wq, w_scales, y, M, N, K, vec, stream);
        else if (rt == 2)
            launch_gemv_rt<2>(y_kind, xq, sx, wq, w_scales, y, M, N, K, vec, stream);
        else
            launch_gemv_rt<4>(y_kind, xq, sx, wq, w_scales, y, M, N, K, vec, stream);
        return hipGetLastError();
    }
    int *partial = sh.split > 1 ? (int *)ws : nullptr;
    hipError_t e;
    if (sh.bm == 256)
        e = launch_tile<256, 256, 2, 4, 2>(y_kind, xq, sx, wq, w_scales, y, partial, M, N, K, sh.split, vec, stream);
    else if (sh.bn == 128)
        e = launch_tile<128, 128, 2, 2, 2>(y_kind, xq, sx, wq, w_scales, y, partial, M, N, K, sh.split, vec, stream);
    else if (sh.bm == 128)
        e = launch_tile<128, 64, 2, 2, 3>(y_kind, xq, sx, wq, w_scales, y, partial, M, N, K, sh.split, vec, stream);
    else
        e = launch_tile<64, 64, 2, 2, 3>(y_kind, xq, sx, wq, w_scales, y, partial, M, N, K, sh.split, vec, stream);
    if (e != hipSuccess || !partial)
        return e;
    const dim3 grid((unsigned)(((M + 15) / 16 * ((N + 15) / 16) + 3) / 4));
    const i32x4 *sums = (const i32x4 *)partial;
    if (y_kind == 2)
        hipLaunchKernelGGL(q4_int8_join_kernel<2>, grid, dim3(256), 0, stream, sums, sx, w_scales, y, M, N, sh.split,
                           vec);
    else if (y_kind == 1)
        hipLaunchKernelGGL(q4_int8_join_kernel<1>, grid, dim3(256), 0, stream, sums, sx, w_scales, y, M, N, sh.split,
                           vec);
    else
        hipLaunchKernelGGL(q4_int8_join_kernel<0>, grid, dim3(256), 0, stream, sums, sx, w_scales, y, M, N, sh.split,
                           vec);
    return hipGetLastError();
}

}  // namespace q4
