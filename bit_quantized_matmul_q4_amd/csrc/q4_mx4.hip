// q4_mx4.hip -- the matrix product in microscaled 4-bit floating point for
// gfx950 (MI355X):
//
//     y[m][n] = sum_b 2^(ex[m][b] + ew[n][b]) sum_{k in b} cx[m][k] cw[n][k]
//
// over blocks b of 32 k (q4_mx4_device.hpp has the form).  The scaled matrix
// instruction v_mfma_scale_f32_16x16x128 takes both operands and their scales
// as they are stored.  A row's sum is one chain of such instructions over its
// steps of 128 k, in order, from +0, in every kernel: its bits depend on the
// row and W alone, not on M, the row's place or the kernel.  A step adds its
// 128 products to the sum with an error of about 2^-24 of the magnitudes that
// it adds; sums of a few thousand products of like size stay exact, since a
// product is a multiple of a quarter of its block's scales.
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
// one row tile by 512 k.
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
                *(u32x4 *)(packed + (tile * steps + step) * 1024 + 16 * lane) = v;
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

// Packed -> values [rows][K], the quantizer's lanes.
template <int KIND>
__global__ __launch_bounds__(256) void q4_mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                                const uint8_t *__restrict__ scales,
                                                                void *__restrict__ y, int rows, int K, unsigned units)
{
    constexpr int SIZE = KIND == 2 ? 4 : 2;
    const int lane = threadIdx.x & 63, p = lane & 15, g = p >> 2;
    const int groups = mx4_groups(K), steps = mx4_steps(K);
    const int c = (threadIdx.x >> 6) * 4 + (lane >> 4);
    for (unsigned unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const size_t tile = unit / groups, row = tile * 16 + c;
        const int group = (int)(unit % groups);
        if (row >= (size_t)rows)
            continue;
        const uint32_t bytes = *(const uint32_t *)(scales + (size_t)unit * 256 + 64 * g + 4 * c);
        uint32_t w[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int step = 4 * group + s;
            w[s] = step < steps
                       ? *(const uint32_t *)(codes + (tile * steps + step) * 1024 + 256 * g + 16 * c + 4 * (p & 3))
                       : 0;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = 512 * group + 128 * s + 8 * p;
            if (k >= K)
                continue;
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = code_value((w[s] >> (4 * i)) & 15, (bytes >> (8 * s)) & 255);
            char *out = (char *)y + (row * K + k) * SIZE;
            if constexpr (KIND == 2) {
                *(f32x4 *)out = (f32x4){f[0], f[1], f[2], f[3]};
                *((f32x4 *)out + 1) = (f32x4){f[4], f[5], f[6], f[7]};
            } else {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = KIND == 1 ? bf16_bits(f[2 * i]) | bf16_bits(f[2 * i + 1]) << 16
                                     : f16_bits(f[2 * i]) | f16_bits(f[2 * i + 1]) << 16;
                *(u32x4 *)out = o;
            }
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

// LDS-tiled: a workgroup of WM x WN waves owns BM rows by BN columns; groups
// of four steps go through LDS one after the other.
template <int BM, int BN, int WM, int WN, int YK>
__global__ __launch_bounds__(64 * WM *WN) void q4_mx4_gemm_kernel(
    const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs, const uint8_t *__restrict__ wq,
    const uint8_t *__restrict__ ws, void *__restrict__ y, int M, int N, int K, int vec)
{
    constexpr int WAVES = WM * WN;
    constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN;
    constexpr int TILES = (BM + BN) / 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[TILES * 4 * 1024];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave % WM, wn = wave / WM;
    const int steps = mx4_steps(K), groups = mx4_groups(K);
    const int tm_all = (M + 15) / 16, tn_all = (N + 15) / 16;
    const int gm = (M + BM - 1) / BM;
    const int bm = blockIdx.x % gm, bn = blockIdx.x / gm;
    const int mt = bm * (BM / 16), nt = bn * (BN / 16);
    f32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
            acc[i][j] = (f32x4){0, 0, 0, 0};
    for (int q = 0; q < groups; ++q) {
        const int here = min(4, steps - 4 * q);
        __syncthreads();
        for (int i = wave; i < TILES * 4; i += WAVES) {
            const int t = i / 4, s = i % 4;
            if (s < here) {
                const bool of_x = t < BM / 16;
                const size_t tile = of_x ? min(mt + t, tm_all - 1) : min(nt + t - BM / 16, tn_all - 1);
                *(u32x4 *)(lds + i * 1024 + lane * 16) =
                    *(const u32x4 *)((of_x ? xq : wq) + (tile * steps + 4 * q + s) * 1024 + lane * 16);
            }
        }
        uint32_t sx[TM], sw[TN];
#pragma unroll
        for (int j = 0; j < TM; ++j)
            sx[j] = *(const uint32_t *)(xs + ((size_t)min(mt + wm * TM + j, tm_all - 1) * groups + q) * 256 + lane * 4);
#pragma unroll
        for (int i = 0; i < TN; ++i)
            sw[i] = *(const uint32_t *)(ws + ((size_t)min(nt + wn * TN + i, tn_all - 1) * groups + q) * 256 + lane * 4);
        __syncthreads();
        const auto step = [&](auto u) {
            if (u.value < here) {
                u32x4 a[TN], b[TM];
#pragma unroll
                for (int j = 0; j < TM; ++j)
                    b[j] = *(const u32x4 *)(lds + ((wm * TM + j) * 4 + u.value) * 1024 + lane * 16);
#pragma unroll
                for (int i = 0; i < TN; ++i)
                    a[i] = *(const u32x4 *)(lds + ((BM / 16 + wn * TN + i) * 4 + u.value) * 1024 + lane * 16);
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = multiply_step<u.value>(a[i], b[j], acc[i][j], sw[i], sx[j]);
            }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
    }
    const int m0 = bm * BM + wm * TM * 16 + (lane & 15), n0 = bn * BN + wn * TN * 16 + 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int m = m0 + 16 * j, n = n0 + 16 * i;
            if (m < M && n < N)
                store4<YK>(y, (size_t)m * N + n, N - n, vec, acc[i][j]);
        }
}

template <int YK>
hipError_t launch_tiles(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, void *y, int M,
                        int N, int K, int vec, hipStream_t stream)
{
    const Mx4Shape sh = mx4_shape(M, N, K);
    const dim3 grid((unsigned)((M + sh.bm - 1) / sh.bm * ((N + sh.bn - 1) / sh.bn)));
    hipLaunchKernelGGL((q4_mx4_gemm_kernel<64, 64, 2, 2, YK>), grid, dim3(256), 0, stream, xq, xs, wq, ws, y, M, N, K,
                       vec);
    return hipGetLastError();
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
    (void)N;
    return dense ? up256(mx4_code_bytes(M, K)) + up256(mx4_scale_bytes(M, K)) : 0;
}

hipError_t launch_mx4_linear(const void *x, int x_kind, const uint8_t *x_scales, const uint8_t *wq, const uint8_t *ws,
                             void *y, int y_kind, int M, int N, int K, void *workspace, hipStream_t stream)
{
    const int size = y_kind == 2 ? 4 : 2;
    const int vec = N % 4 == 0 && ((uintptr_t)y & (4 * size - 1)) == 0;
    const uint8_t *xq = (const uint8_t *)x, *xs = x_scales;
    if (x_kind >= 0) {
        uint8_t *q = (uint8_t *)workspace, *s = q + up256(mx4_code_bytes(M, K));
        const hipError_t e = launch_mx4_quantize(x, x_kind, q, s, true, M, K, stream);
        if (e != hipSuccess)
            return e;
        xq = q;
        xs = s;
    }
    if (y_kind == 2)
        return launch_tiles<2>(xq, xs, wq, ws, y, M, N, K, vec, stream);
    if (y_kind == 1)
        return launch_tiles<1>(xq, xs, wq, ws, y, M, N, K, vec, stream);
    return launch_tiles<0>(xq, xs, wq, ws, y, M, N, K, vec, stream);
}

}  // namespace q4
