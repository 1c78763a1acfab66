// q4_probe.hip -- probe kernels for the GPU tests and the benchmark's
// calibration read (libq4probe.so).
//
// They run the library's own device primitives (q4_device.hpp) on raw lane
// data so the tests can check, on the hardware, the assumptions the fixed
// reduction order rests on: the MFMA operand / result lane layout, that an
// MFMA result element depends only on its own A row and B column (not on its
// slot or on other rows), run-to-run determinism, the nibble dequantization
// and the corrected block dot.  Not part of the product library.
//
// probe_issue times a wave's block dots, FMAs, or both interleaved, for
// the benchmark's check of how far the matrix core and the VALU overlap.
//
// probe_read is a plain streaming read of a device buffer: the benchmark's
// yardstick of the bandwidth the memory system delivers to a simple kernel
// ("a big copy, not the spec sheet", in "Why LLM Decoding Is Slow, and Why
// Batching Is (Almost) Free", section "First Attempt: A Faster Chip").
//
// probe_ring_read reads with the matrix-vector kernels' streaming structure
// and nothing else: each wave streams its own contiguous run of 1 KB quads
// (16 bytes a lane, non-temporal) through a D-deep register ring, in
// workgroups of a given number of waves; the benchmark's floor for a kernel
// of that structure.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_device.hpp"
#include "q4_int8_plan.hpp"
#include "q4_moe_plan.hpp"

namespace {

// One MFMA per wave: a, b are [waves][64 lanes][4 dwords], d is [waves][64][4].
template <bool BF16>
__global__ __launch_bounds__(64) void probe_mfma(const q4::u32x4 *a, const q4::u32x4 *b, q4::f32x4 *d)
{
    const int i = blockIdx.x * 64 + threadIdx.x;
    d[i] = q4::blockdot<BF16>(a[i], b[i]);
}

template <bool BF16>
__global__ __launch_bounds__(256) void probe_dequant(const uint32_t *w, q4::u32x4 *out, int n)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        out[i] = q4::Dequant<BF16>()(w[i]);
}

// One MFMA per wave with the accumulator input c: d = MFMA(a, b, C = c).
template <bool BF16>
__global__ __launch_bounds__(64) void probe_mfma_acc(const q4::u32x4 *a, const q4::u32x4 *b, const q4::f32x4 *c,
                                                     q4::f32x4 *d)
{
    const int i = blockIdx.x * 64 + threadIdx.x;
    d[i] = q4::blockdot_acc<BF16>(a[i], b[i], c[i]);
}

// The block dot of the order as the kernels run it: for lane data a (A
// operand) and one packed code word w per lane, the correction C = MFMA(a,
// -24) (bf16) or 0 (fp16) and the block dot D = MFMA(a, dequant(w), C = C)
// (bf16) or MFMA(a, dequant(w)) (fp16); both are returned, [waves][64][4]
// each.
template <bool BF16>
__global__ __launch_bounds__(64) void probe_q4dot(const q4::u32x4 *a, const uint32_t *w, q4::f32x4 *d,
                                                  q4::f32x4 *e)
{
    const int i = blockIdx.x * 64 + threadIdx.x;
    const q4::Dequant<BF16> dq;
    const q4::f32x4 c = q4::correction<BF16>(a[i], dq);
    d[i] = q4::block_dot<BF16>(a[i], dq(w[i]), c);
    e[i] = c;
}

// fmaf(d, s, +0) on the VALU, for the single-rounding check of the scale step.
__global__ __launch_bounds__(256) void probe_fma0(const float *d, const float *s, float *out, int n)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        out[i] = __builtin_fmaf(d[i], s[i], 0.0f);
}

// Grid-stride 16-byte non-temporal loads, eight in flight per thread; the
// xor of everything read goes to sink[0] only if it equals a value no real
// buffer is known to give, so the loads cannot be dropped and nothing else
// is written.  n16: number of 16-byte words.
__global__ __launch_bounds__(512) void probe_read(const q4::u32x4 *__restrict__ src, size_t n16, uint32_t *sink)
{
    const size_t stride = (size_t)gridDim.x * blockDim.x;
    size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    q4::u32x4 acc = {0u, 0u, 0u, 0u};
    for (; i + 7 * stride < n16; i += 8 * stride) {
        q4::u32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = __builtin_nontemporal_load(src + i + u * stride);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            acc ^= v[u];
    }
    for (; i < n16; i += stride)
        acc ^= __builtin_nontemporal_load(src + i);
    const uint32_t r = acc.x ^ acc.y ^ acc.z ^ acc.w;
    if (r == 0x9E3779B9u)
        sink[0] = r;
}

// Wave w (of W) streams quads w Q .. w Q + Q - 1 (1 KB each, lane l reading
// bytes 16 l .. 16 l + 15) with D loads in flight; refills past the run read
// its last quad again (in range).  The xor of everything read goes to
// sink[0] only if it equals a value no real buffer is known to give.
template <int D>
__global__ __launch_bounds__(1024) void probe_ring_read(const q4::u32x4 *__restrict__ src, int Q, int W,
                                                        uint32_t *sink)
{
    const int lane = threadIdx.x & 63;
    const int w = blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    if (w >= W)
        return;
    const q4::u32x4 *run = src + (size_t)w * Q * 64 + lane;
    q4::u32x4 r[D];
#pragma unroll
    for (int u = 0; u < D; ++u)
        r[u] = __builtin_nontemporal_load(run + 64 * (size_t)min(u, Q - 1));
    q4::u32x4 acc = {0u, 0u, 0u, 0u};
    for (int q = 0; q < Q; q += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            acc ^= r[u];
            r[u] = __builtin_nontemporal_load(run + 64 * (size_t)min(q + u + D, Q - 1));
        }
    }
#pragma unroll
    for (int u = 0; u < D; ++u)
        acc ^= r[u];
    const uint32_t v = acc.x ^ acc.y ^ acc.z ^ acc.w;
    if (v == 0x9E3779B9u)
        sink[0] = v;
}

// Issue-overlap probe: per iteration a wave runs 4 independent bf16 block
// dots (v_mfma_f32_16x16x32_bf16 into 4 accumulators) when MODE & 1 and 16
// independent fp32 FMAs (8 chains) when MODE & 2, so the time of MODE 3
// against MODES 1 and 2 tells whether the matrix core and the VALU of the
// waves on a SIMD work in parallel.  One value per thread goes to out (so
// nothing is dropped).
template <int MODE>
__global__ __launch_bounds__(256) void probe_issue(float *out, int iters, float s)
{
    const int t = threadIdx.x;
    const q4::u32x4 a = {0x3F803F80u + t, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const q4::u32x4 b = {0x3F803F80u, 0x3F803F80u + t, 0x3F803F80u, 0x3F803F80u};
    q4::f32x4 c0 = {0.f, 0.f, 0.f, 0.f}, c1 = c0, c2 = c0, c3 = c0;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = (float)(t + j);
    for (int i = 0; i < iters; ++i) {
        if constexpr ((MODE & 1) != 0) {
            const q4::bf16x8 A = __builtin_bit_cast(q4::bf16x8, a), B = __builtin_bit_cast(q4::bf16x8, b);
            c0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B, c0, 0, 0, 0);
            c1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B, c1, 0, 0, 0);
            c2 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B, c2, 0, 0, 0);
            c3 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B, c3, 0, 0, 0);
        }
        if constexpr ((MODE & 2) != 0) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = __builtin_fmaf(v[j], s, 1.0f);
        }
        asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]),
                     "+v"(v[7]));
    }
    float r = c0.x + c1.y + c2.z + c3.w;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        r += v[j];
    out[blockIdx.x * 256 + t] = r;
}

// An empty kernel (one store that never happens): the benchmark's measure of
// the fixed cost of one launch in a graph.
__global__ __launch_bounds__(256) void probe_empty(uint32_t *sink, int v)
{
    if (v == 0x5EED && threadIdx.x == 0)
        sink[blockIdx.x] = (uint32_t)v;
}

}  // namespace

extern "C" {

// `blocks` workgroups of 256 threads that do nothing (sink is never written
// for v != 0x5EED; it must hold `blocks` words if v == 0x5EED).
int q4probe_empty(void *sink, int blocks, int v, void *stream)
{
    if (!sink || blocks < 1)
        return -1;
    hipLaunchKernelGGL(probe_empty, dim3(blocks), dim3(256), 0, (hipStream_t)stream, (uint32_t *)sink, v);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

// The issue-overlap probe (mode 1: block dots only, 2: FMAs only, 3: both)
// with `blocks` workgroups of 4 waves; out holds 256 blocks floats.
int q4probe_issue(int mode, void *out, int blocks, int iters, void *stream)
{
    if (!out || blocks < 1 || iters < 1 || mode < 1 || mode > 3)
        return -1;
    hipStream_t st = (hipStream_t)stream;
    if (mode == 1)
        hipLaunchKernelGGL(probe_issue<1>, dim3(blocks), dim3(256), 0, st, (float *)out, iters, 0.5f);
    else if (mode == 2)
        hipLaunchKernelGGL(probe_issue<2>, dim3(blocks), dim3(256), 0, st, (float *)out, iters, 0.5f);
    else
        hipLaunchKernelGGL(probe_issue<3>, dim3(blocks), dim3(256), 0, st, (float *)out, iters, 0.5f);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

// Streams `bytes` (a multiple of 16, src 16-byte aligned) with `blocks`
// workgroups of 512 threads.
int q4probe_read(const void *src, size_t bytes, void *sink, int blocks, void *stream)
{
    if (!src || !sink || bytes % 16 || blocks < 1)
        return -1;
    hipLaunchKernelGGL(probe_read, dim3(blocks), dim3(512), 0, (hipStream_t)stream, (const q4::u32x4 *)src,
                       bytes / 16, (uint32_t *)sink);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

// Reads waves x quads KB from src (16-byte aligned) with the streaming
// structure of probe_ring_read: workgroups of waves_per_group (1..16) waves,
// depth 2 or 4.
int q4probe_ring_read(const void *src, int quads, int waves, int waves_per_group, int depth, void *sink,
                      void *stream)
{
    if (!src || !sink || quads < 1 || waves < 1 || waves_per_group < 1 || waves_per_group > 16 ||
        (depth != 2 && depth != 4))
        return -1;
    const dim3 grid((unsigned)((waves + waves_per_group - 1) / waves_per_group)), block(64u * waves_per_group);
    if (depth == 2)
        hipLaunchKernelGGL(probe_ring_read<2>, grid, block, 0, (hipStream_t)stream, (const q4::u32x4 *)src, quads,
                           waves, (uint32_t *)sink);
    else
        hipLaunchKernelGGL(probe_ring_read<4>, grid, block, 0, (hipStream_t)stream, (const q4::u32x4 *)src, quads,
                           waves, (uint32_t *)sink);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int q4probe_mfma_acc(const void *a, const void *b, const void *c, void *d, int waves, int bf16, void *stream)
{
    if (!a || !b || !c || !d || waves < 1)
        return -1;
    if (bf16)
        hipLaunchKernelGGL(probe_mfma_acc<true>, dim3(waves), dim3(64), 0, (hipStream_t)stream,
                           (const q4::u32x4 *)a, (const q4::u32x4 *)b, (const q4::f32x4 *)c, (q4::f32x4 *)d);
    else
        hipLaunchKernelGGL(probe_mfma_acc<false>, dim3(waves), dim3(64), 0, (hipStream_t)stream,
                           (const q4::u32x4 *)a, (const q4::u32x4 *)b, (const q4::f32x4 *)c, (q4::f32x4 *)d);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int q4probe_mfma(const void *a, const void *b, void *d, int waves, int bf16, void *stream)
{
    if (!a || !b || !d || waves < 1)
        return -1;
    if (bf16)
        hipLaunchKernelGGL(probe_mfma<true>, dim3(waves), dim3(64), 0, (hipStream_t)stream,
                           (const q4::u32x4 *)a, (const q4::u32x4 *)b, (q4::f32x4 *)d);
    else
        hipLaunchKernelGGL(probe_mfma<false>, dim3(waves), dim3(64), 0, (hipStream_t)stream,
                           (const q4::u32x4 *)a, (const q4::u32x4 *)b, (q4::f32x4 *)d);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int q4probe_dequant(const void *w, void *out, int n, int bf16, void *stream)
{
    if (!w || !out || n < 1)
        return -1;
    const dim3 grid((n + 255) / 256);
    if (bf16)
        hipLaunchKernelGGL(probe_dequant<true>, grid, dim3(256), 0, (hipStream_t)stream,
                           (const uint32_t *)w, (q4::u32x4 *)out, n);
    else
        hipLaunchKernelGGL(probe_dequant<false>, grid, dim3(256), 0, (hipStream_t)stream,
                           (const uint32_t *)w, (q4::u32x4 *)out, n);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int q4probe_q4dot(const void *a, const void *w, void *d, void *e, int waves, int bf16, void *stream)
{
    if (!a || !w || !d || !e || waves < 1)
        return -1;
    if (bf16)
        hipLaunchKernelGGL(probe_q4dot<true>, dim3(waves), dim3(64), 0, (hipStream_t)stream,
                           (const q4::u32x4 *)a, (const uint32_t *)w, (q4::f32x4 *)d, (q4::f32x4 *)e);
    else
        hipLaunchKernelGGL(probe_q4dot<false>, dim3(waves), dim3(64), 0, (hipStream_t)stream,
                           (const q4::u32x4 *)a, (const uint32_t *)w, (q4::f32x4 *)d, (q4::f32x4 *)e);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int q4probe_fma0(const void *d, const void *s, void *out, int n, void *stream)
{
    if (!d || !s || !out || n < 1)
        return -1;
    hipLaunchKernelGGL(probe_fma0, dim3((n + 255) / 256), dim3(256), 0, (hipStream_t)stream,
                       (const float *)d, (const float *)s, (float *)out, n);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

// The form of the 8-bit product that a shape takes, for the tests that name
// what they run (host only): {quantized within the product, one column tile a
// workgroup, rows and columns of the tile, split of K, rows a workgroup of the
// quantizer}.
int q4probe_int8_form(int dense, int M, int N, int K, int *form)
{
    const q4::Int8Shape s = q4::int8_shape(dense != 0, M, N, K);
    form[0] = s.decode;
    form[1] = s.gemv;
    form[2] = s.bm;
    form[3] = s.bn;
    form[4] = s.split;
    form[5] = q4::quant_rows(M);
    return 0;
}

// The same for the expert layer: {experts chosen within gate/up, logits by
// rows}.
int q4probe_moe_form(int M, int E, int H, int *form)
{
    form[0] = q4::moe_fused(M, E, H);
    form[1] = q4::moe_by_rows(M, E, H);
    return 0;
}

}  // extern "C"
