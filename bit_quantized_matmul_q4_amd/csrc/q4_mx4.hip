// q4_mx4.hip -- the matrix product in microscaled 4-bit floating point for
// gfx950 (MI355X):
//
//     y[m][n] = sum_b 2^(ex[m][b] + ew[n][b]) sum_{k in b} cx[m][k] cw[n][k]
//
// over blocks b of 32 k (q4_mx4_device.hpp has the form).  The scaled matrix
// instruction v_mfma_scale_f32_16x16x128 takes both operands and their scales
// as they are stored.  A row's sum is one chain of such instructions over its
// steps of 128 k, in order, from +0, in every kernel: its bits depend on the
// row and W alone, not on M, the row's place or the kernel.  A step adds its four
// blocks one after another, each exactly and then within 2^-23 of the sum's size;
// a block all of whose products stand 2^28 or more below the sum is lost (measured:
// 1 and 128 products of 36 2^-32 give 1, 18 2^-24 off).  Sums of a few thousand products
// of like size stay exact, since a product is a multiple of a quarter of its
// block's scales.
//
// Packed layout of both operands (q4.h): codes in tiles of 16 rows by 128 k,
// order [ceil(rows / 16)][ceil(K / 128)], 1024 bytes each; lane l = 16 g + c
// of a wave owns bytes 16 l .. 16 l + 15: row 16 t + c, the block k = 128 q +
// 32 g .. + 31, even k in the low half of a byte.  Scale bytes in tiles of 16
// rows by 512 k, 256 bytes each; lane l owns bytes 4 l .. 4 l + 3, its block's
// in four steps.  That is the instruction's operand order, so a wave's loads
// from memory and from LDS are contiguous and need no swizzle.  Entries past
// the rows or past K are zero.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "q4_launch.hpp"
#include "q4_mx4_device.hpp"

namespace q4 {

namespace {

using namespace mx4;

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ------------------------------------------------------------- quantizer
// A workgroup takes 16 rows by 512 k, a wave four of the rows: 16 lanes a row
// and step of 128 k, eight values a lane, so that a block is a quad of lanes.
// A lane with the first part of a block ends with its bytes of four steps.
// Bound by the reads: 18944 x 3584 packed from binary32 in 56 to 58 us a replayed
// call (5.3 to 5.5 TB/s read and written; 53 under a tracer, which leaves out the
// time between two kernels), from bfloat16 in 32 (5.4); to the canonical form 59
// and 33.  Binary32 in whole lines a load (four values a lane, a block eight
// lanes) took 57.7 where this took 57.6.
// PACKED: the packed form (padding written), else codes [rows][K / 2] and
// scales [rows][K / 32].
template <int KIND, bool PACKED>
__global__ __launch_bounds__(256) void q4_mx4_quantize_kernel(const void *__restrict__ x_, uint8_t *__restrict__ codes,
                                                              uint8_t *__restrict__ scales, int rows, int K,
                                                              unsigned units)
{
    constexpr int VECS = kVecs<KIND>, SIZE = KIND == 2 ? 4 : 2;
    const int lane = threadIdx.x & 63, p = lane & 15, g = p >> 2;
    const int groups = mx4_groups(K), steps = mx4_steps(K);
    const int c = (threadIdx.x >> 6) * 4 + (lane >> 4);
    for (unsigned unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const size_t tile = unit / groups, row = tile * 16 + c;
        const int group = (int)(unit % groups);
        const bool live = row < (size_t)rows;
        const char *x = (const char *)x_ + (live ? row : 0) * K * SIZE;
        u32x4 v[4][VECS];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = 512 * group + 128 * s + 8 * p;
#pragma unroll
            for (int i = 0; i < VECS; ++i)
                v[s][i] = live && k < K ? *((const u32x4 *)(x + (size_t)k * SIZE) + i) : (u32x4){0, 0, 0, 0};
        }
        uint32_t bytes = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int step = 4 * group + s, k = 128 * step + 8 * p;
            const uint32_t byte = scale_byte(top_of_quad(top8<KIND>(v[s])));
            const uint32_t w = codes8<KIND>(v[s], byte);
            bytes |= byte << (8 * s);
            if constexpr (PACKED) {
                if (step < steps)
                    *(uint32_t *)(codes + (tile * steps + step) * 1024 + 256 * g + 16 * c + 4 * (p & 3)) = w;
            } else if (live && k < K) {
                *(uint32_t *)(codes + row * (K / 2) + k / 2) = w;
                if ((p & 3) == 0)
                    scales[row * (K / 32) + k / 32] = (uint8_t)byte;
            }
        }
        if (PACKED && (p & 3) == 0)
            *(uint32_t *)(scales + (size_t)unit * 256 + 64 * g + 4 * c) = bytes;
    }
}

// Canonical codes [rows][K / 2] and scales [rows][K / 32] -> packed; a wave
// one row tile by 512 k.  18944 x 3584 in 14.5 us (5.0 TB/s read and written;
// with stores that are to be kept 20.7).
__global__ __launch_bounds__(256) void q4_mx4_pack_kernel(const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales,
                                                          uint8_t *__restrict__ packed, uint8_t *__restrict__ tiles,
                                                          int rows, int K, unsigned units)
{
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int groups = mx4_groups(K), steps = mx4_steps(K);
    for (unsigned unit = blockIdx.x * 4 + (threadIdx.x >> 6); unit < units; unit += 4 * gridDim.x) {
        const size_t tile = unit / groups, row = tile * 16 + c;
        const int group = (int)(unit % groups);
        uint32_t bytes = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int step = 4 * group + s, k = 128 * step + 32 * g;
            u32x4 v = {0, 0, 0, 0};
            if (row < (size_t)rows && k < K) {
                v = *(const u32x4 *)(codes + row * (K / 2) + k / 2);
                bytes |= (uint32_t)scales[row * (K / 32) + k / 32] << (8 * s);
            }
            if (step < steps)
                __builtin_nontemporal_store(v, (u32x4 *)(packed + (tile * steps + step) * 1024 + 16 * lane));
        }
        *(uint32_t *)(tiles + (size_t)unit * 256 + 4 * lane) = bytes;
    }
}

// ------------------------------------------------------- values and outputs
__device__ __forceinline__ uint32_t bf16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t f16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// The value of a code times a scale, rounded once where binary32 cannot hold
// it (an infinity past its largest).
__device__ __forceinline__ float code_value(uint32_t code, uint32_t byte)
{
    const uint32_t e = (code >> 1) & 3, m = code & 1;
    const float size = e ? __builtin_bit_cast(float, (e + 126) << 23 | m << 22) : 0.5f * (float)m;
    const float v = __builtin_ldexpf(size, (int)byte - 127);
    return byte == 255 ? __builtin_nanf("") : code & 8 ? -v : v;
}

// Packed -> values [rows][K]: 16 lanes a row and step of 128 k, as the
// quantizer, 16 bytes a lane and store, so that a store fills whole lines.  Bound
// by the stores, which are marked as not to be kept: 18944 x 3584 to bfloat16
// took 43 us with ordinary ones, 33 so (5.2 TB/s); to binary32, with a lane's
// eight values in two stores of which each fills half of every line, 79 and 109
// us, in whole lines 50 (6.1 TB/s): codes from the last-level cache, where the
// quantizer leaves them; from memory they are 35 and 62 us.
template <int KIND>
__global__ __launch_bounds__(256) void q4_mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                                const uint8_t *__restrict__ scales,
                                                                void *__restrict__ y, int rows, int K, unsigned units)
{
    constexpr int SIZE = KIND == 2 ? 4 : 2, PER = 16 / SIZE, PARTS = 8 / PER;  // values a store, stores a step
    typedef std::conditional_t<KIND == 2, uint16_t, uint32_t> Codes;           // PER of them
    const int lane = threadIdx.x & 63, p = lane & 15;
    const int groups = mx4_groups(K), steps = mx4_steps(K);
    const int c = (threadIdx.x >> 6) * 4 + (lane >> 4);
    for (unsigned unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const size_t tile = unit / groups, row = tile * 16 + c;
        const int group = (int)(unit % groups);
        if (row >= (size_t)rows)
            continue;
        uint32_t bytes[PARTS], w[4][PARTS];
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
            const int k = PER * (16 * i + p);  // in its step
            bytes[i] = *(const uint32_t *)(scales + (size_t)unit * 256 + k / 32 * 64 + 4 * c);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int step = min(4 * group + s, steps - 1);
                w[s][i] =
                    *(const Codes *)(codes + (tile * steps + step) * 1024 + k / 32 * 256 + 16 * c + k % 32 / 2);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const int k = 512 * group + 128 * s + PER * (16 * i + p);
                if (k >= K)
                    continue;
                float f[PER];
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    f[e] = code_value((w[s][i] >> (4 * e)) & 15, (bytes[i] >> (8 * s)) & 255);
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = KIND == 2   ? __builtin_bit_cast(uint32_t, f[e])
                           : KIND == 1 ? bf16_bits(f[2 * e % PER]) | bf16_bits(f[(2 * e + 1) % PER]) << 16
                                       : f16_bits(f[2 * e % PER]) | f16_bits(f[(2 * e + 1) % PER]) << 16;
                __builtin_nontemporal_store(o, (u32x4 *)((char *)y + (row * K + k) * SIZE));
            }
    }
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
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = YK == 1 ? bf16_bits(v[i]) : f16_bits(v[i]);
        if (vec && left >= 4) {
            *(uint2 *)p = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left)
                    p[i] = (uint16_t)h[i];
        }
    }
}

// One step of the chain: 16 columns of W by 16 rows of x over 128 k, with the
// scale bytes U of both words.  Lane (g, c) holds row c of x, columns 4 g .. 4
// g + 3 of W.
template <int U>
__device__ __forceinline__ f32x4 multiply_step(u32x4 w, u32x4 x, f32x4 acc, uint32_t ws, uint32_t xs)
{
    const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 b = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, U, (int)ws, U, (int)xs);
}

// -------------------------------------------------------------- the product
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t src, uint8_t *lds, int lane_at, int at)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void *)lds, 16, lane_at, at, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N < 63 ? N : 63) : "memory");
}

// Which tile a workgroup takes: workgroups go to the 8 dies in turn; each die
// takes a run of tiles, in bands of eight row tiles, so that few panels of x
// and W pass through its L2 at once (4096 x 18944 x 3584 with four 146.5 us, with
// eight 145.3).
struct TileAt {
    int bm, bn;
};
__device__ __forceinline__ TileAt tile_at(int id, int gm, int gn)
{
    const int total = gm * gn, q = total / 8, r = total % 8, die = id & 7;
    id = die * q + min(die, r) + (id >> 3);
    const int band = id / (8 * gn), rows_in = min(8, gm - 8 * band), in_band = id - 8 * band * gn;
    return TileAt{8 * band + in_band % rows_in, in_band / rows_in};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t *p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), (short)0, bytes, 0x00020000);
}

// Lane (g, c) holds row c of a tile of x, columns 4 g .. 4 g + 3 of one of W.
template <int TM, int TN, int YK>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[TN][TM], void *y, int m0, int n0, int M, int N, int vec)
{
    const int lane = threadIdx.x & 63;
    m0 += lane & 15;
    n0 += 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int m = m0 + 16 * j, n = n0 + 16 * i;
            if (m < M && n < N)
                store4<YK>(y, (size_t)m * N + n, N - n, vec, acc[i][j]);
        }
}

// The lane, made anew: what is computed from it is not held in registers over
// the products.
__device__ __forceinline__ int fresh_lane()
{
    int lane;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
    return lane;
}

// Writes to LDS as instructions of their own: the compiler would wait for every
// load and store in flight before each, since loads into LDS might go to the
// same place.
__device__ __forceinline__ void lds_write(uint8_t *p, u32x4 v)
{
    asm volatile("ds_write_b128 %0, %1" ::"v"((__attribute__((address_space(3))) uint8_t *)p), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_write(uint8_t *p, uint2 v)
{
    asm volatile("ds_write_b64 %0, %1" ::"v"((__attribute__((address_space(3))) uint8_t *)p),
                 "v"((uint64_t)v.y << 32 | v.x)
                 : "memory");
}

// Sixteen bytes at any address of their elements' alignment.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// 16 rows by 64 columns of a wave's tile, by way of LDS (4 KB of the wave's
// own): whole rows of 128 bytes (256 in binary32) leave together.  A row's
// 16-byte pieces lie in an order of its own, so that neither the writes (16
// rows at once) nor the reads meet in a bank.  The stores are marked as not
// to be kept: 4096 x 18944 x 3584 took 163 us with ordinary ones against 146,
// and 181 with each lane's own four columns.  ALL: no row or column is past
// the end.
template <int YK, bool ALL>
__device__ __forceinline__ void store_rows(const f32x4 (&v)[4], uint8_t *l, void *y, int m0, int n0, int M, int N)
{
    constexpr int SIZE = YK == 2 ? 4 : 2, PIECE = 16 / SIZE, P = 64 / PIECE;  // P pieces a row
    constexpr int R = 64 / P, STORES = 16 / R;                              // R rows a store
    const int lane = fresh_lane(), c = lane & 15, g = lane >> 4;
    if constexpr (YK == 2) {
        // (the sums come from matrix instructions, which the compiler does not
        // wait for before an instruction of ours)
        f32x4 w[4] = {v[0], v[1], v[2], v[3]};
        asm volatile("s_nop 15\n\ts_nop 15" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            lds_write(l + c * 256 + ((4 * i + g) ^ c) * 16, __builtin_bit_cast(u32x4, w[i]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h[e] = YK == 1 ? bf16_bits(v[i][e]) : f16_bits(v[i][e]);
            lds_write(l + c * 128 + ((2 * i + g / 2) ^ (c & 7)) * 16 + g % 2 * 8,
                      make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16));
        }
    }
    const int piece = lane % P, r0 = lane / P;
    u32x4 o[STORES];
#pragma unroll
    for (int r = 0; r < STORES; ++r)
        o[r] = *(const u32x4 *)(l + (R * r + r0) * 16 * P + (piece ^ ((R * r + r0) & (P - 1))) * 16);
    const int left = N - n0 - PIECE * piece;
    char *out = (char *)y + ((size_t)(m0 + r0) * N + n0 + PIECE * piece) * SIZE;
#pragma unroll
    for (int r = 0; r < STORES; ++r) {
        if (ALL || (m0 + R * r + r0 < M && left >= PIECE)) {
            __builtin_nontemporal_store(o[r], (u32x4_any *)out);
        } else if (m0 + R * r + r0 < M) {
#pragma unroll
            for (int i = 0; i < PIECE; ++i)
                if (i < left) {
                    if constexpr (YK == 2)
                        ((uint32_t *)out)[i] = o[r][i];
                    else
                        ((uint16_t *)out)[i] = (uint16_t)(o[r][i / 2] >> (16 * (i & 1)));
                }
        }
        out += (size_t)R * N * SIZE;
    }
}

// Few rows, at most 16: bound by the bytes of W.
constexpr int kFewWaves = 4, kFewSteps = 8;
constexpr uint32_t kNowhere = 1u << 31;  // past every tile's range: reads zero, no access

// Rows of x into LDS by the whole workgroup: [step][block of the step][row]
// codes, 16 bytes each, then [group][block of a step][row] the scale bytes of
// four steps (mx4_few_lds bytes).  KIND 0, 1: dense rows, quantized on the way;
// -1: packed rows.
template <int KIND>
__device__ __forceinline__ void stage_rows(uint8_t *lds, const void *x_, const uint8_t *xs, int M, int K)
{
    constexpr int THREADS = 64 * kFewWaves, HELD = 4;
    const int steps = mx4_steps(K), groups = mx4_groups(K);
    uint8_t *const lds_s = lds + steps * 64 * M;
    // items of a row, and what divides by them (exact below 2^32 / items)
    const int items = KIND < 0 ? M : steps * 16, all = KIND < 0 ? steps * 4 * M : M * items;
    const uint32_t inverse = (uint32_t)((0x100000000ull + items - 1) / items);
    const auto quotient = [&](int i) { return items == 1 ? i : (int)__umulhi((uint32_t)i, inverse); };
    for (int i0 = threadIdx.x; i0 < all; i0 += HELD * THREADS) {
        u32x4 v[HELD][1];
        int row[HELD], k[HELD];
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const int i = i0 + h * THREADS, q = quotient(i), r = i - q * items;
            if constexpr (KIND < 0) {  // (a block's 16 bytes, as packed)
                row[h] = r;
                k[h] = 32 * q;
                v[h][0] = i < all ? *(const u32x4 *)((const uint8_t *)x_ + 256 * q + 16 * r) : (u32x4){0, 0, 0, 0};
            } else {
                row[h] = q;
                k[h] = 8 * r;
                v[h][0] = i < all && k[h] < K ? *(const u32x4 *)((const uint16_t *)x_ + (size_t)q * K + k[h])
                                              : (u32x4){0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            uint8_t *const at = lds + (k[h] / 32 * M + row[h]) * 16;
            if constexpr (KIND < 0) {
                if (i0 + h * THREADS < all)
                    *(u32x4 *)at = v[h][0];
            } else {
                const uint32_t byte = scale_byte(top_of_quad(top8<KIND>(v[h])));
                const uint32_t w = codes8<KIND>(v[h], byte);
                if (i0 + h * THREADS < all) {
                    *(uint32_t *)(at + k[h] % 32 / 2) = w;
                    if (k[h] % 32 == 0)
                        lds_s[((k[h] / 512 * 4 + k[h] / 32 % 4) * M + row[h]) * 4 + k[h] / 128 % 4] = (uint8_t)byte;
                }
            }
        }
    }
    if constexpr (KIND < 0)
        for (int i = threadIdx.x; i < groups * 4 * M; i += THREADS) {
            const int q = quotient(i), r = i - q * M;
            *(uint32_t *)(lds_s + 4 * i) = *(const uint32_t *)(xs + 64 * q + 4 * r);
        }
}

// A run of steps of a tile of W and their scale bytes (past the end: zeros);
// X: with the rows' own.
template <bool X>
struct Run {
    u32x4 w[kFewSteps], x[X ? kFewSteps : 1];
    uint32_t ws[kFewSteps / 4], xs[X ? kFewSteps / 4 : 1];
};
__device__ __forceinline__ u32x4 load_codes(__amdgpu_buffer_rsrc_t b, int s, int steps, int at)
{
    return __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, s < steps ? s * 1024 + at * 16 : kNowhere, 0, 0));
}
__device__ __forceinline__ uint32_t load_bytes(__amdgpu_buffer_rsrc_t b, int q, int groups, int at)
{
    return __builtin_amdgcn_raw_buffer_load_b32(b, q < groups ? q * 256 + at * 4 : kNowhere, 0, 0);
}
template <bool X>
__device__ __forceinline__ void load_run(Run<X> &r, __amdgpu_buffer_rsrc_t wb, __amdgpu_buffer_rsrc_t wsb, int s0,
                                         int steps, int groups)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u)
        r.w[u] = load_codes(wb, s0 + u, steps, lane);
#pragma unroll
    for (int u = 0; u < kFewSteps / 4; ++u)
        r.ws[u] = load_bytes(wsb, s0 / 4 + u, groups, lane);
}
__device__ __forceinline__ void load_rows(Run<true> &r, __amdgpu_buffer_rsrc_t xb, __amdgpu_buffer_rsrc_t xsb, int s0,
                                          int steps, int groups, int at)
{
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u)
        r.x[u] = load_codes(xb, s0 + u, steps, at);
#pragma unroll
    for (int u = 0; u < kFewSteps / 4; ++u)
        r.xs[u] = load_bytes(xsb, s0 / 4 + u, groups, at);
}
// acc goes on by the run's steps; x: their operands, from LDS all at once where
// the run does not hold them.
template <bool X>
__device__ __forceinline__ f32x4 multiply_run(const Run<X> &r, f32x4 acc, const uint8_t *lds, int s0, int steps, int M)
{
    const int lane = threadIdx.x & 63, g = lane >> 4, c = min(lane & 15, M - 1);
    const uint8_t *const lds_s = lds + steps * 64 * M;
    u32x4 x[kFewSteps];
    uint32_t xs[kFewSteps / 4];
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u)
        x[u] = X ? r.x[X ? u : 0] : *(const u32x4 *)(lds + ((min(s0 + u, steps - 1) * 4 + g) * M + c) * 16);
#pragma unroll
    for (int u = 0; u < kFewSteps / 4; ++u)
        xs[u] = X ? r.xs[X ? u : 0]
                  : *(const uint32_t *)(lds_s + ((min(s0 + 4 * u, steps - 1) / 4 * 4 + g) * M + c) * 4);
    const auto step = [&](auto u) {
        if (s0 + u.value < steps)
            acc = multiply_step<u.value & 3>(r.w[u.value], x[u.value], acc, r.ws[u.value / 4], xs[u.value / 4]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    step(std::integral_constant<int, 4>{});
    step(std::integral_constant<int, 5>{});
    step(std::integral_constant<int, 6>{});
    step(std::integral_constant<int, 7>{});
    return acc;
}

// A workgroup owns 16 columns.  Its waves hold runs of W in registers, two
// ahead, and hand the sums on from wave to wave by way of LDS, so that the
// chain keeps its order while every wave's loads are in flight.  Dense rows
// stand in LDS; packed ones are loaded beside W (staged like the dense ones they
// took 5.5 us at 16 x 3584 x 3584, beside W 4.2).  Bound by the launch and the
// loads' latency, or W's bytes: 1 x 3584 x 3584 with the quantization 5.0 us, 8 x
// 18944 x 3584 on packed rows 9.5 (3.8 TB/s; 8.4 with W in the last-level cache).
template <int KIND, int YK>
__global__ __launch_bounds__(64 * kFewWaves) void q4_mx4_relay_kernel(const void *__restrict__ x,
                                                                      const uint8_t *__restrict__ xs,
                                                                      const uint8_t *__restrict__ wq,
                                                                      const uint8_t *__restrict__ ws,
                                                                      void *__restrict__ y, int M, int N, int K,
                                                                      int vec)
{
    constexpr int U = kFewSteps, W = kFewWaves;
    constexpr bool X = KIND < 0;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ f32x4 sum[64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int steps = mx4_steps(K), groups = mx4_groups(K);
    const auto wb = resource(wq + (size_t)blockIdx.x * steps * 1024, steps * 1024);
    const auto wsb = resource(ws + (size_t)blockIdx.x * groups * 256, groups * 256);
    const auto xb = resource((const uint8_t *)x, X ? steps * 1024 : 0), xsb = resource(xs, X ? groups * 256 : 0);
    const int at = (lane & 48) + min(lane & 15, M - 1);
    Run<X> r0, r1;
    const auto load = [&](Run<X> &r, int s0) {
        if (s0 < steps) {
            load_run(r, wb, wsb, s0, steps, groups);
            if constexpr (X)
                load_rows(r, xb, xsb, s0, steps, groups, at);
        }
    };
    load(r0, wave * U);
    load(r1, (W + wave) * U);
    if constexpr (!X)
        stage_rows<KIND>(lds, x, xs, M, K);
    sum[lane] = (f32x4){0, 0, 0, 0};
    __syncthreads();
    const auto round = [&](Run<X> &r, int s0) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (wave == w && s0 + w * U < steps) {
                sum[lane] = multiply_run(r, sum[lane], lds, s0 + w * U, steps, M);
                load(r, s0 + (2 * W + w) * U);
            }
            __syncthreads();
        }
    };
    for (int s0 = 0; s0 < steps; s0 += 2 * W * U) {
        round(r0, s0);
        if (s0 + W * U < steps)
            round(r1, s0 + W * U);
    }
    if (wave == 0) {
        const int m = lane & 15, n = 16 * blockIdx.x + 4 * (lane >> 4);
        if (m < M && n < N)
            store4<YK>(y, (size_t)m * N + n, N - n, vec, sum[lane]);
    }
}

// Many columns: a wave owns 16 at a time, two runs of W ahead of the products
// (the next tile's included), with the rows in LDS; workgroups as many as stay
// on the card.  Bound by W's bytes: 1 x 152064 x 896 in 14.6 us (5.0 TB/s), 1 x 65536 x
// 3584 in 22.7 (5.5).
template <int KIND, int YK>
__global__ __launch_bounds__(64 * kFewWaves) void q4_mx4_wide_kernel(const void *__restrict__ x,
                                                                     const uint8_t *__restrict__ xs,
                                                                     const uint8_t *__restrict__ wq,
                                                                     const uint8_t *__restrict__ ws,
                                                                     void *__restrict__ y, int M, int N, int K,
                                                                     int vec)
{
    constexpr int U = kFewSteps;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int steps = mx4_steps(K), groups = mx4_groups(K), tiles = (N + 15) / 16;
    const int stride = gridDim.x * kFewWaves;
    int tile = blockIdx.x * kFewWaves + wave, s0 = 0;  // of the run that is multiplied
    int ahead = tile, s1 = 0;                          // of the run that is loaded
    const auto load = [&](Run<false> &r) {
        if (ahead < tiles) {
            load_run(r, resource(wq + (size_t)ahead * steps * 1024, steps * 1024),
                     resource(ws + (size_t)ahead * groups * 256, groups * 256), s1, steps, groups);
            s1 += U;
            if (s1 >= steps) {
                s1 = 0;
                ahead += stride;
            }
        }
    };
    Run<false> r0, r1;
    load(r0);
    load(r1);
    stage_rows<KIND>(lds, x, xs, M, K);
    __syncthreads();
    f32x4 acc = {0, 0, 0, 0};
    const auto go = [&](Run<false> &r) {
        acc = multiply_run(r, acc, lds, s0, steps, M);
        load(r);
        s0 += U;
        if (s0 >= steps) {
            const int m = lane & 15, n = 16 * tile + 4 * (lane >> 4);
            if (m < M && n < N)
                store4<YK>(y, (size_t)m * N + n, N - n, vec, acc);
            acc = (f32x4){0, 0, 0, 0};
            s0 = 0;
            tile += stride;
        }
    };
    while (tile < tiles) {
        go(r0);
        if (tile < tiles)
            go(r1);
    }
}

// Many rows: a workgroup of four waves owns 128 rows by 256 columns, a wave 128
// by 64.  Steps of x go from memory to LDS directly, three deep, for all
// waves; a wave's own steps of W go to its registers, three ahead, and the scale bytes
// of four steps to LDS with every fourth.  So neither LDS (both operands by way
// of it: as many cycles as the products) nor the vector cache holds up the
// matrix cores, and two workgroups share a compute unit, one's start and end
// beside the other's products.  A wave reads the operands of a step from LDS
// while it multiplies the one before: the barrier that frees a step's place
// falls when its operands are in registers.  4096 x 18944 x 3584 to bfloat16 takes
// 153 to 155 us with operands from memory and 133 with operands in the last-level
// cache (3.6 and 4.2 PF/s; from registers alone the matrix cores reach 6.9); so
// measured, without the stores 126, without W's loads too 105, the products alone 91.
// 256 x 256 with both operands in LDS, in workgroups that stay and take tile
// after tile, took 148, W two steps ahead instead of three 145.
template <int YK>
__global__ __launch_bounds__(256, 2) void q4_mx4_gemm_kernel(
    const void *__restrict__ xq_, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ wq,
    const uint8_t *__restrict__ ws, void *__restrict__ y, int M, int N, int K, int)
{
    constexpr int WN = 4;                        // waves
    constexpr int AHEAD = 3, NS = 3;             // steps of W and of x that come in meanwhile
    constexpr int TM = 8, TN = 4, TW = TN * WN;  // row tiles of x; a wave's and all of W
    constexpr int PER = TM / WN;                 // pieces of x a wave loads a step
    constexpr int STAGE = TM * 1024;
    constexpr int SC = (TM + TW + 4 * WN - 1) / (4 * WN);  // loads of scale bytes a wave: four tiles each
    static_assert(TM % WN == 0 && TN + PER <= TM, "a load between every two rows of products");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    uint8_t *const lds_s = lds + NS * STAGE;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint8_t *const xq = (const uint8_t *)xq_;
    const int steps = mx4_steps(K), groups = mx4_groups(K);
    const int tm_all = (M + 15) / 16, tn_all = (N + 15) / 16;
    const TileAt t = tile_at(blockIdx.x, (M + 127) / 128, (N + 16 * TW - 1) / (16 * TW));
    const int mt = t.bm * TM, nt = t.bn * TW;
    // (row tiles past the end: the last one, its outputs are not stored)
    const int xt = min(tm_all - mt, TM), wt = min(tn_all - nt, TW);
    const auto xb = resource(xq + (size_t)mt * steps * 1024, xt * steps * 1024);
    const auto wb = resource(wq + (size_t)nt * steps * 1024, wt * steps * 1024);
    const auto xsb = resource(xs + (size_t)mt * groups * 256, xt * groups * 256);
    const auto wsb = resource(ws + (size_t)nt * groups * 256, wt * groups * 256);
    int at[PER], at_w[TN], at_s[SC];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        at[i] = min(i * WN + wave, xt - 1) * steps * 1024;
#pragma unroll
    for (int i = 0; i < TN; ++i)
        at_w[i] = min(wave * TN + i, wt - 1) * steps * 1024;
#pragma unroll
    for (int i = 0; i < SC; ++i) {
        const int first = 4 * (i * WN + wave);
        const int tile = min((first < TM ? first : first - TM) + lane / 16, (first < TM ? xt : wt) - 1);
        at_s[i] = tile * groups * 256 + lane % 16 * 16;
    }
    // (past the last step: the last again, so that the counts of loads stay)
    const int last = (steps - 1) * 1024, last_s = (groups - 1) * 256;
    int to = 0, from = 0, next = 0, next_s = 0;  // places in LDS to fill and to read, steps and scale bytes to load
    const auto fetch = [&](int i) {
        load_lds(xb, lds + to + (i * WN + wave) * 1024, lane * 16, at[i] + min(next, last));
    };
    const auto fetched = [&] {
        to = to + STAGE == NS * STAGE ? 0 : to + STAGE;
        next += 1024;
    };
    const auto fetch_scales = [&] {
#pragma unroll
        for (int i = 0; i < SC; ++i)
            load_lds(4 * (i * WN + wave) < TM ? xsb : wsb, lds_s + (i * WN + wave) * 1024, at_s[i],
                     min(next_s, last_s));
        next_s += 256;
    };
    f32x4 acc[TN][TM];
    u32x4 a[4][TN], b[TM];
    uint32_t sw[TN], sw_next[TN], sx[TM];
    const auto load_w = [&](int to, int i, int s) {
        a[to][i] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(wb, lane * 16, at_w[i] + min(s * 1024, last), 0));
    };
    const auto read_x = [&](int j) { b[j] = *(const u32x4 *)(lds + from + j * 1024 + lane * 16); };
    const auto read_xs = [&](int j) { sx[j] = *(const uint32_t *)(lds_s + j * 256 + lane * 4); };
    const auto read_ws = [&](int i) {
        return *(const uint32_t *)(lds_s + (TM + wave * TN + i) * 256 + lane * 4);
    };
    // (W's last step ahead between the pieces of x, as later on, so that one count
    // of loads holds for every step)
    const auto load_step = [&](int s) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
            load_w(s, i, s);
    };
    const auto fetch_step = [&] {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            fetch(i);
        fetched();
    };
    fetch_scales();
    load_step(0);
    load_step(1);
    __builtin_amdgcn_sched_barrier(0);
    fetch_step();
    __builtin_amdgcn_sched_barrier(0);
    fetch_step();
    __builtin_amdgcn_sched_barrier(0);
    load_step(2);
    __builtin_amdgcn_sched_barrier(0);
    fetch_step();
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<2 * PER + TN>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        read_x(j);
        read_xs(j);
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        sw[i] = read_ws(i);
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = (f32x4){0, 0, 0, 0};
    }
    // Step s, U-th of its group: its operands are in registers.  Wait for the next
    // step's pieces of x (and the next group's scale bytes), and let this step's
    // place go.  The scale bytes' place is read at a group's start and filled again
    // after its first step.  Loads and reads stand between the products, which go
    // on meanwhile.  (Past the last step: what is read is not used.)  END, the
    // steps after the last whole group: no step is three later, W has arrived or is on
    // its way, and none of its loads counts (loads that nothing uses are not there).
    const auto step = [&](auto u, auto end, int s) {
        constexpr int U = u.value;
        constexpr bool END = end.value;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_loads<PER + (END ? 0 : TN) + (U == 1 || U == 2 ? SC : 0)>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        from = from + STAGE == NS * STAGE ? 0 : from + STAGE;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < TN; ++i)
                acc[i][j] = multiply_step<U>(a[U][i], b[j], acc[i][j], sw[i], sx[j]);
            __builtin_amdgcn_sched_barrier(0);
            read_x(j);
            if constexpr (U == 3) {
                read_xs(j);
                if (j < TN)
                    sw_next[j] = read_ws(j);
            }
            if (j < TN && !END)
                load_w((U + AHEAD) & 3, j, s + AHEAD);
            else if (j >= TN && j - TN < PER)
                fetch(j - TN);
            if (U == 0 && j == TM - 1)
                fetch_scales();
        }
        __builtin_amdgcn_sched_barrier(0);
        fetched();
        if constexpr (U == 3) {
#pragma unroll
            for (int i = 0; i < TN; ++i)
                sw[i] = sw_next[i];
        }
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 3> I3;
    int s = 0;
#pragma clang loop unroll(disable)
    for (; s + 4 <= steps; s += 4) {  // (no branch: the compiler counts the loads in flight)
        step(I0{}, std::false_type{}, s);
        step(I1{}, std::false_type{}, s + 1);
        step(I2{}, std::false_type{}, s + 2);
        step(I3{}, std::false_type{}, s + 3);
    }
    if (s < steps) {
        step(I0{}, std::true_type{}, s);
        if (s + 1 < steps)
            step(I1{}, std::true_type{}, s + 1);
        if (s + 2 < steps)
            step(I2{}, std::true_type{}, s + 2);
    }
    // (what was loaded past the end is in place before LDS holds outputs)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int m0 = t.bm * 128, n0 = (nt + wave * TN) * 16;
    const bool all = m0 + 16 * TM <= M && n0 + 16 * TN <= N;
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        f32x4 v[TN];
#pragma unroll
        for (int i = 0; i < TN; ++i)
            v[i] = acc[i][j];
        if (all)
            store_rows<YK, true>(v, lds + wave * 4096, y, m0 + 16 * j, n0, M, N);
        else
            store_rows<YK, false>(v, lds + wave * 4096, y, m0 + 16 * j, n0, M, N);
    }
}

// Some rows: a workgroup of WN waves owns 16 TM rows by 16 TN WN columns, a
// wave all of the rows by 16 TN.  Groups of four steps of x and their scale
// bytes go from memory to LDS directly, A + 1 deep, for all waves; a wave's own
// steps of W go to its registers, A groups ahead.  A wave reads the operands
// of a step from LDS while it multiplies the one before; the one barrier of a
// group stands before its last products, when their operands are in registers.
// Bound by the chain of groups (a barrier, LDS and dependent products each) and
// by what passes through L2 (x for each column of tiles, W for each row):
// 124 x 3584 x 18944 in 19.4 us on 224 workgroups of 32 x 64, 0.52 us a group, and 124 x
// 18944 x 3584 in 16.2 on 148 of 128 x 128, with W from memory (13.6, 0.37 a group, and
// 13.5 with W in the last-level cache).
template <int TM, int TN, int WN, int A, int YK>
__global__ __launch_bounds__(64 * WN) void q4_mx4_mid_kernel(
    const void *__restrict__ xq_, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ wq,
    const uint8_t *__restrict__ ws, void *__restrict__ y, int M, int N, int K, int vec)
{
    constexpr int TW = TN * WN, NS = A + 1;
    static_assert(A % 2 == 0);
    static_assert(4 * TM % WN == 0, "every wave loads as many pieces of x");
    constexpr int PER = 4 * TM / WN, SX = (TM + 3) / 4, SC = (SX + WN - 1) / WN;
    constexpr int STAGE = TM * 4096 + SC * WN * 1024;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint8_t *const xq = (const uint8_t *)xq_;
    const int steps = mx4_steps(K), groups = mx4_groups(K);
    const int tm_all = (M + 15) / 16, tn_all = (N + 15) / 16;
    const TileAt t = tile_at(blockIdx.x, (M + 16 * TM - 1) / (16 * TM), (N + 16 * TW - 1) / (16 * TW));
    const int mt = t.bm * TM, nt = t.bn * TW;
    // (row tiles past the end: the last one, its outputs are not stored)
    const int xt = min(tm_all - mt, TM), wt = min(tn_all - nt, TW);
    const auto xb = resource(xq + (size_t)mt * steps * 1024, xt * steps * 1024);
    const auto wb = resource(wq + (size_t)nt * steps * 1024, wt * steps * 1024);
    const auto xsb = resource(xs + (size_t)mt * groups * 256, xt * groups * 256);
    const auto wsb = resource(ws + (size_t)nt * groups * 256, wt * groups * 256);
    // (past the last step or group: the last again, so that the counts stay)
    int to = 0;  // the place of the next group to come in
    const auto fetch = [&](int group) {
        const int q = min(group, groups - 1);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int piece = i * WN + wave, tile = min(piece / 4, xt - 1), step = min(4 * q + piece % 4, steps - 1);
            load_lds(xb, lds + to + piece * 1024, lane * 16, (tile * steps + step) * 1024);
        }
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            const int piece = i * WN + wave, tile = min(4 * min(piece, SX - 1) + lane / 16, xt - 1);
            load_lds(xsb, lds + to + TM * 4096 + piece * 1024, tile * groups * 256 + lane % 16 * 16, q * 256);
        }
        to = to + STAGE == NS * STAGE ? 0 : to + STAGE;
    };
    int at_w[TN], at_s[TN];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
        at_w[i] = min(wave * TN + i, wt - 1) * steps * 1024;
        at_s[i] = min(wave * TN + i, wt - 1) * groups * 256;
    }
    u32x4 a[A][4][TN], b[2][TM];
    uint32_t sw[A][TN], sx[2][TM];
    const auto load_w = [&](auto buf, auto u, int q) {
        const int s = min(4 * q + u.value, steps - 1) * 1024;
#pragma unroll
        for (int i = 0; i < TN; ++i)
            a[buf.value][u.value][i] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(wb, lane * 16, at_w[i] + s, 0));
    };
    const auto load_ws = [&](auto buf, int q) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
            sw[buf.value][i] =
                __builtin_amdgcn_raw_buffer_load_b32(wsb, lane * 4, at_s[i] + min(q, groups - 1) * 256, 0);
    };
    int from = 0;  // the place of the group that is read
    const auto read_x = [&](int to, int u) {
#pragma unroll
        for (int j = 0; j < TM; ++j)
            b[to][j] = *(const u32x4 *)(lds + from + (j * 4 + u) * 1024 + lane * 16);
    };
    const auto read_xs = [&](int to) {
#pragma unroll
        for (int j = 0; j < TM; ++j)
            sx[to][j] = *(const uint32_t *)(lds + from + TM * 4096 + j * 256 + lane * 4);
    };
    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = (f32x4){0, 0, 0, 0};
    const auto multiply = [&](auto buf, auto u) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int i = 0; i < TN; ++i)
                acc[i][j] = multiply_step<u.value>(a[buf.value][u.value][i], b[u.value & 1][j], acc[i][j],
                                                   sw[buf.value][i], sx[buf.value & 1][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 3> I3;
    // (in the order of the loop, so that one count of loads holds for every group)
    load_w(I0{}, I0{}, 0);
    load_w(I0{}, I1{}, 0);
    load_w(I0{}, I2{}, 0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(1);
    const auto begin = [&](auto buf, auto next) {
        __builtin_amdgcn_sched_barrier(0);
        load_w(buf, I3{}, buf.value);
        load_ws(buf, buf.value);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (next.value < A) {
            load_w(next, I0{}, next.value);
            load_w(next, I1{}, next.value);
            load_w(next, I2{}, next.value);
            __builtin_amdgcn_sched_barrier(0);
            fetch(next.value + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    begin(I0{}, I1{});
    begin(I1{}, I2{});
    if constexpr (A == 4) {
        begin(I2{}, I3{});
        begin(I3{}, std::integral_constant<int, 4>{});
    }
    wait_loads<A *(PER + SC) + (A - 1) * 5 * TN + 2 * TN>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read_x(0, 0);
    read_xs(0);
    // END, the groups from which none is A later: no loads of W, and none of them
    // counts (loads that nothing uses are not there)
    const auto group = [&](auto buf, auto other, auto end, int q) {
        constexpr bool END = end.value;
        const auto load = [&](auto u) {
            if constexpr (!END)
                load_w(buf, u, q + A);
        };
        read_x(1, 1);
        multiply(buf, I0{});
        load(I0{});
        read_x(0, 2);
        multiply(buf, I1{});
        load(I1{});
        read_x(1, 3);
        multiply(buf, I2{});
        load(I2{});
        // every wave is done with this group's place, and the next group is here
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_loads<(NS - 2) * (PER + SC) + (END ? 0 : (NS - 1) * 5 * TN)>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fetch(q + NS);
        from = from + STAGE == NS * STAGE ? 0 : from + STAGE;
        read_x(0, 0);
        read_xs(other.value & 1);
        multiply(buf, I3{});
        load(I3{});
        if constexpr (!END)
            load_ws(buf, q + A);
    };
    const auto last = [&](auto buf, int q) {  // of one to four steps
        read_x(1, 1);
        multiply(buf, I0{});
        read_x(0, 2);
        if (4 * q + 1 < steps)
            multiply(buf, I1{});
        read_x(1, 3);
        if (4 * q + 2 < steps)
            multiply(buf, I2{});
        if (4 * q + 3 < steps)
            multiply(buf, I3{});
    };
    int q = 0;
#pragma clang loop unroll(disable)
    for (; q + A < groups; q += A) {  // (no branch: the compiler counts the loads in flight)
        group(I0{}, I1{}, std::false_type{}, q);
        group(I1{}, std::integral_constant<int, 2 % A>{}, std::false_type{}, q + 1);
        if constexpr (A == 4) {
            group(I2{}, I3{}, std::false_type{}, q + 2);
            group(I3{}, I0{}, std::false_type{}, q + 3);
        }
    }
    const auto end = [&](auto buf, auto other) {  // false: the last group
        if (q + buf.value + 1 == groups) {
            last(buf, q + buf.value);
            return false;
        }
        group(buf, other, std::true_type{}, q + buf.value);
        return true;
    };
    if (end(I0{}, I1{}) && end(I1{}, std::integral_constant<int, 2 % A>{})) {
        if constexpr (A == 4) {
            if (end(I2{}, I3{}))
                end(I3{}, I0{});
        }
    }
    wait_loads<0>();  // (the loads past the end: nothing is in flight into LDS when the workgroup ends)
    store_tile<TM, TN, YK>(acc, y, t.bm * 16 * TM, (nt + wave * TN) * 16, M, N, vec);
}

// An entry point's pointers and sizes, as the kernels take them.
struct Args {
    const void *x;
    const uint8_t *xs, *wq, *ws;
    void *y;
    int M, N, K, vec;
};

unsigned tile_count(const Args &a, int bm, int bn) { return (unsigned)mx4_tile_count(a.M, a.N, bm, bn); }

template <typename Kernel>
hipError_t launch(Kernel kernel, unsigned grid, int waves, int lds, const Args &a, hipStream_t stream)
{
    if (lds > 64 * 1024) {
        const hipError_t e =
            hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * waves), lds, stream, a.x, a.xs, a.wq, a.ws, a.y, a.M, a.N, a.K,
                       a.vec);
    return hipGetLastError();
}

template <int KIND, int YK>
hipError_t launch_few(const Args &a, Mx4Kernel kernel, hipStream_t stream)
{
    const unsigned tiles = tile_count(a, 16, 16);
    const int lds = mx4_few_lds(a.M, a.K);
    if (kernel == Mx4Kernel::wide)
        return launch(q4_mx4_wide_kernel<KIND, YK>, std::min((tiles + 3) / 4, 2u * kMx4Units), kFewWaves, lds, a,
                      stream);
    return launch(q4_mx4_relay_kernel<KIND, YK>, tiles, kFewWaves, KIND < 0 ? 0 : lds, a, stream);
}

template <int TM, int TN, int WN, int A, int YK>
hipError_t launch_mid(const Args &a, hipStream_t stream)
{
    constexpr int kLds = (A + 1) * (TM * 4096 + ((TM + 3) / 4 + WN - 1) / WN * WN * 1024);
    return launch(q4_mx4_mid_kernel<TM, TN, WN, A, YK>, tile_count(a, 16 * TM, 16 * TN * WN), WN, kLds, a, stream);
}

template <int YK>
hipError_t launch_product(int x_kind, Mx4Kernel kernel, const Args &a, hipStream_t stream)
{
    switch (kernel) {
    case Mx4Kernel::relay:
    case Mx4Kernel::wide:
        return x_kind < 0    ? launch_few<-1, YK>(a, kernel, stream)
               : x_kind == 1 ? launch_few<1, YK>(a, kernel, stream)
                             : launch_few<0, YK>(a, kernel, stream);
    case Mx4Kernel::tile16x32: return launch_mid<1, 1, 2, 4, YK>(a, stream);
    case Mx4Kernel::tile32x32: return launch_mid<2, 1, 2, 2, YK>(a, stream);
    case Mx4Kernel::tile32x64: return launch_mid<2, 1, 4, 2, YK>(a, stream);
    case Mx4Kernel::tile64x64: return launch_mid<4, 1, 4, 2, YK>(a, stream);
    case Mx4Kernel::tile64x128: return launch_mid<4, 2, 4, 2, YK>(a, stream);
    case Mx4Kernel::tile128x128: return launch_mid<8, 2, 4, 2, YK>(a, stream);
    case Mx4Kernel::tile128x256: break;
    }
    constexpr int kIn = 3 * 8 * 1024 + 2 * 4 * 1024;  // x's steps and the scale bytes, then the outputs' rows
    return launch(q4_mx4_gemm_kernel<YK>, tile_count(a, 128, 256), 4, kIn, a, stream);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Row tiles times groups of 512 k: a workgroup each, up to 2^20 of them (so
// that a launch stays below 2^32 threads), which go on in steps of that.
unsigned tile_groups(int rows, int K) { return (unsigned)((rows + 15) / 16) * (unsigned)mx4_groups(K); }
dim3 unit_grid(unsigned units) { return dim3(std::min(units, 1u << 20)); }

}  // namespace

size_t mx4_code_bytes(int rows, int K) { return (size_t)((rows + 15) / 16) * mx4_steps(K) * 1024; }
size_t mx4_scale_bytes(int rows, int K) { return (size_t)((rows + 15) / 16) * mx4_groups(K) * 256; }

hipError_t launch_mx4_quantize(const void *x, int kind, uint8_t *codes, uint8_t *scales, bool packed, int rows, int K,
                               hipStream_t stream)
{
    const unsigned units = tile_groups(rows, K);
    const dim3 grid = unit_grid(units), block(256);
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, x, codes, scales, rows, K, units);
        return hipGetLastError();
    };
    if (packed)
        return kind == 2   ? go(q4_mx4_quantize_kernel<2, true>)
               : kind == 1 ? go(q4_mx4_quantize_kernel<1, true>)
                           : go(q4_mx4_quantize_kernel<0, true>);
    return kind == 2   ? go(q4_mx4_quantize_kernel<2, false>)
           : kind == 1 ? go(q4_mx4_quantize_kernel<1, false>)
                       : go(q4_mx4_quantize_kernel<0, false>);
}

hipError_t launch_mx4_pack(const uint8_t *codes, const uint8_t *scales, uint8_t *packed, uint8_t *tiles, int rows,
                           int K, hipStream_t stream)
{
    const unsigned units = tile_groups(rows, K);
    hipLaunchKernelGGL(q4_mx4_pack_kernel, unit_grid((units + 3) / 4), dim3(256), 0, stream, codes, scales, packed,
                       tiles, rows, K, units);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, void *y, int kind, int rows, int K,
                                 hipStream_t stream)
{
    const unsigned units = tile_groups(rows, K);
    const dim3 grid = unit_grid(units), block(256);
    if (kind == 2)
        hipLaunchKernelGGL(q4_mx4_dequantize_kernel<2>, grid, block, 0, stream, codes, scales, y, rows, K, units);
    else if (kind == 1)
        hipLaunchKernelGGL(q4_mx4_dequantize_kernel<1>, grid, block, 0, stream, codes, scales, y, rows, K, units);
    else
        hipLaunchKernelGGL(q4_mx4_dequantize_kernel<0>, grid, block, 0, stream, codes, scales, y, rows, K, units);
    return hipGetLastError();
}

size_t mx4_workspace_bytes(bool dense, int M, int N, int K)
{
    return dense && !mx4_shape(true, M, N, K).fused ? up256(mx4_code_bytes(M, K)) + up256(mx4_scale_bytes(M, K)) : 0;
}

hipError_t launch_mx4_linear(const void *x, int x_kind, const uint8_t *x_scales, const uint8_t *wq, const uint8_t *ws,
                             void *y, int y_kind, int M, int N, int K, void *workspace, hipStream_t stream)
{
    const int size = y_kind == 2 ? 4 : 2;
    const int vec = N % 4 == 0 && ((uintptr_t)y & (4 * size - 1)) == 0;
    Args a{x, x_scales, wq, ws, y, M, N, K, vec};
    const Mx4Shape sh = mx4_shape(x_kind >= 0, M, N, K);
    if (x_kind >= 0 && !sh.fused) {
        uint8_t *q = (uint8_t *)workspace, *s = q + up256(mx4_code_bytes(M, K));
        const hipError_t e = launch_mx4_quantize(x, x_kind, q, s, true, M, K, stream);
        if (e != hipSuccess)
            return e;
        a.x = q;
        a.xs = s;
        x_kind = -1;
    }
    if (y_kind == 2)
        return launch_product<2>(x_kind, sh.kernel, a, stream);
    if (y_kind == 1)
        return launch_product<1>(x_kind, sh.kernel, a, stream);
    return launch_product<0>(x_kind, sh.kernel, a, stream);
}

}  // namespace q4
