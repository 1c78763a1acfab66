// q4_norm.hip -- what stands between two linear layers of a block, in one
// pass over the rows, for gfx950 (MI355X):
//
//     r[m] = residual[m] + scale gate[m] post(y[m])
//     h[m] = pre(r[m])
//
// post and pre are norms (or none):
//     rms    v / sqrt(mean(v^2) + eps) weight + bias
//     layer  (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) weight + bias
// Everything between the loads and the stores is binary32 (a mean's sum
// binary64): pre sees r before it is rounded to its stored type, and h is
// rounded once, to a float type or to the packed microscaled 4-bit form
// (q4_mx4_device.hpp).
//
// A workgroup owns a row and holds it in registers, eight neighbouring values
// a lane and piece, so that every value is read and written once.  The shape
// of the sums is a function of H alone: a row's bits depend on neither M nor
// the row's place.  A sum of squares that leaves binary32's range is taken
// again on values divided by a power of two (normalize).
//
// Many rows are bound by their bytes: 4096 x 3584, y binary32, residual, gate, r
// and h bfloat16, with both norms, takes 40.3 us (4.4 TB/s read and written; a
// copy of 2 GiB 4.9).  Few are bound by the launch and one latency of memory
// after another (the row, post's weight, pre's): 1 x 3584 takes 3.8 us, 333 x
// 4863, whose rows start at odd elements, 10.0 (4864: 9.3).  Fetching a
// line of each weight at the start cost 0.2 to 1 us there.  Stores that are not
// to be kept took 38.9 us instead of 40.5 at 4096 x 3584, but the product and the
// norm that read r and h next lost more than that (80.6 against 78.2 for all
// three).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_launch.hpp"
#include "q4_mx4_device.hpp"

namespace q4 {

namespace {

using namespace mx4;

// Sixteen bytes at any address of their elements' alignment.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// Eight values as loaded: binary32 in both vectors, 16-bit types in the first.
struct Raw {
    u32x4 v[2];
};

// Values at .. at + 7 of an array of a type (0 binary16, 1 bfloat16, 2
// binary32), those from `left` on zero.  A row's last values come one by one,
// all of them on their way at once.
__device__ __forceinline__ Raw load8(const void *p, int kind, size_t at, int left)
{
    Raw r = {{{0, 0, 0, 0}, {0, 0, 0, 0}}};
    if (left >= 8) {
        if (kind == 2) {
            r.v[0] = *(const u32x4_any *)((const float *)p + at);
            r.v[1] = *(const u32x4_any *)((const float *)p + at + 4);
        } else {
            r.v[0] = *(const u32x4_any *)((const uint16_t *)p + at);
        }
    } else if (left > 0) {
        uint32_t d[8];
        if (kind == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = ((const uint32_t *)p)[at + min(i, left - 1)];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r.v[i / 4][i % 4] = i < left ? d[i] : 0;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = ((const uint16_t *)p)[at + min(i, left - 1)];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r.v[0][i / 2] |= (i < left ? d[i] : 0) << (16 * (i & 1));
        }
    }
    return r;
}

__device__ __forceinline__ void values8(const Raw &r, int kind, float (&f)[8])
{
    if (kind == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __builtin_bit_cast(float, (uint32_t)r.v[i / 4][i % 4]);
    } else if (kind == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __builtin_bit_cast(float, i & 1 ? r.v[0][i / 2] & 0xFFFF0000u : r.v[0][i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = (float)__builtin_bit_cast(f16x2, (uint32_t)r.v[0][i / 2])[i & 1];
    }
}

__device__ __forceinline__ void store8(void *p, int kind, size_t at, int left, const float (&f)[8])
{
    if (kind == 2) {
        float *o = (float *)p + at;
        if (left >= 8) {
            u32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __builtin_bit_cast(uint32_t, f[i]);
                b[i] = __builtin_bit_cast(uint32_t, f[i + 4]);
            }
            *(u32x4_any *)o = a;
            *(u32x4_any *)(o + 4) = b;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left)
                    o[i] = f[i];
        }
        return;
    }
    uint16_t *o = (uint16_t *)p + at;
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kind == 1)
            w[i] = __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
        else
            w[i] = __builtin_bit_cast(uint32_t, (f16x2){(_Float16)f[2 * i], (_Float16)f[2 * i + 1]});
    }
    if (left >= 8) {
        *(u32x4_any *)o = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left)
                o[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

// Sum of a wave's lanes, in every lane: neighbours within 16, then the four 16s.
__device__ __forceinline__ float lanes(float v, int l)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
template <int CTRL>
__device__ __forceinline__ float moved(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
typedef int i32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ double lanes(double v, int l)
{
    const i32x2 w = __builtin_bit_cast(i32x2, v);
    return __builtin_bit_cast(double, (i32x2){__builtin_amdgcn_readlane(w.x, l), __builtin_amdgcn_readlane(w.y, l)});
}
template <int CTRL>
__device__ __forceinline__ double moved(double v)
{
    const i32x2 w = __builtin_bit_cast(i32x2, v);
    return __builtin_bit_cast(double, (i32x2){__builtin_amdgcn_mov_dpp(w.x, CTRL, 0xF, 0xF, true),
                                              __builtin_amdgcn_mov_dpp(w.y, CTRL, 0xF, 0xF, true)});
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v)
{
    v += moved<0xB1>(v);   // lanes 1 0 3 2
    v += moved<0x4E>(v);   // lanes 2 3 0 1
    v += moved<0x141>(v);  // eight mirrored
    v += moved<0x140>(v);  // sixteen mirrored
    return (lanes(v, 0) + lanes(v, 16)) + (lanes(v, 32) + lanes(v, 48));
}
__device__ __forceinline__ float wave_max(float v)
{
    v = __builtin_fmaxf(v, moved<0xB1>(v));
    v = __builtin_fmaxf(v, moved<0x4E>(v));
    v = __builtin_fmaxf(v, moved<0x141>(v));
    v = __builtin_fmaxf(v, moved<0x140>(v));
    return __builtin_fmaxf(__builtin_fmaxf(lanes(v, 0), lanes(v, 16)), __builtin_fmaxf(lanes(v, 32), lanes(v, 48)));
}

// What the waves of a row pass to each other in one norm: each use has a place
// of its own, so that one barrier is enough.
constexpr int kMaxWaves = 16;
struct Parts {
    double sum[kMaxWaves];
    float square[kMaxWaves], top[kMaxWaves];
};

// Sum over the row's T threads, the same bits in each: within the waves, then
// the waves in order.
template <int T, typename V>
__device__ __forceinline__ V row_sum(V v, V *part)
{
    v = wave_sum(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w)
            v += part[w];
    }
    return v;
}
template <int T>
__device__ __forceinline__ float row_max(float v, float *part)
{
    v = wave_max(v);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
            part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w)
            v = __builtin_fmaxf(v, part[w]);
    }
    return v;
}

// The row's mean (0 for rms) as a binary32 number and what that is off by, and
// the mean square about both.  The mean is summed in binary64, where a sum of
// equal values is exact, and what is left about its binary32 number comes from
// the sum itself: in a row of equal values every difference is 0, and in one
// of nearly equal values none is more than a few roundings of its own off.
// Values past H are zero and stay out of the squares.
struct Moments {
    float mean, rest, square;
};

template <int T, int C>
__device__ __forceinline__ Moments moments(float (&v)[C][8], bool layer, int H, Parts &part)
{
    float mean = 0.f, rest = 0.f;
    if (layer) {
        const double count = (double)H, over = 1.0 / count;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float *f = v[i];
            s += (((double)f[0] + (double)f[1]) + ((double)f[2] + (double)f[3])) +
                 (((double)f[4] + (double)f[5]) + ((double)f[6] + (double)f[7]));
        }
        s = row_sum<T>(s, part.sum);
        mean = (float)(s * over);
        rest = (float)(__builtin_fma(-count, (double)mean, s) * over);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = 8 * ((int)threadIdx.x + i * T);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = at + e < H ? (v[i][e] - mean) - rest : 0.f;
            s = __builtin_fmaf(d, d, s);
        }
    }
    return Moments{mean, rest, row_sum<T>(s, part.square) * (1.f / (float)H)};
}

// v := the norm of v before weight and bias.  Where the sums leave binary32's
// range (a value over 2^63 or so, or an eps next to the largest number; or all
// so small that their squares vanish, and eps no larger), the row is divided by
// the power of two of its largest value first, and the root is taken in binary64.  Infinities and NaN take the
// plain way: finite values over an infinite root are 0.
template <int T, int C>
__device__ __forceinline__ void normalize(float (&v)[C][8], int kind, float eps, int H, Parts &part)
{
    const bool layer = kind == 2;
    Moments m = moments<T, C>(v, layer, H, part);
    const float under = m.square + eps;
    float inv = 1.f / __builtin_sqrtf(under);
    if (!(under < __builtin_inff()) || (m.square < 0x1p-80f && eps < 0x1p-40f)) {
        float top = 0.f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                top = __builtin_fmaxf(top, __builtin_fabsf(v[i][e]));
                nan |= v[i][e] != v[i][e];
            }
        top = row_max<T>(nan ? __builtin_inff() : top, part.top);
        if (top > 0.f && top < __builtin_inff()) {
            const int k = __builtin_amdgcn_frexp_expf(top);
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[i][e] = __builtin_ldexpf(v[i][e], -k);
            __syncthreads();  // (the first sums are read)
            m = moments<T, C>(v, layer, H, part);
            inv = (float)(1.0 / __builtin_sqrt((double)m.square + __builtin_ldexp((double)eps, -2 * k)));
            // (past binary32 only where all values are equal, since others differ by
            // 2^-25 or more here: 0 by a finite number, and 0 / 0 where eps is 0)
            if (eps > 0.f)
                inv = __builtin_fminf(inv, 0x1.fffffep127f);
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = ((v[i][e] - m.mean) - m.rest) * inv;
}

// v := v weight + bias at the thread's pieces.
template <int T, int C>
__device__ __forceinline__ void affine(float (&v)[C][8], const NormSide &n, int H)
{
    Raw w[C], b[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = 8 * ((int)threadIdx.x + i * T);
        if (n.weight)
            w[i] = load8(n.weight, n.type, at, H - at);
        if (n.bias)
            b[i] = load8(n.bias, n.type, at, H - at);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        float f[8];
        if (n.weight) {
            values8(w[i], n.type, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] *= f[e];
        }
        if (n.bias) {
            values8(b[i], n.type, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] += f[e];
        }
    }
}

// One row a workgroup of T threads, C pieces of eight values a thread.
template <int T, int C>
__global__ __launch_bounds__(T) void q4_block_norm_kernel(const NormArgs a)
{
    __shared__ Parts part[2];  // post's and pre's
    const int H = a.H, tid = threadIdx.x;
    const size_t row = blockIdx.x;
    if (row >= (size_t)a.M) {  // a padding row of the packed form
        for (int k = 8 * tid; k < mx4_groups(H) * 512; k += 8 * T) {
            if (k < mx4_steps(H) * 128)
                *(uint32_t *)((uint8_t *)a.h + mx4_code_at(row, k, H)) = 0;
            if (k % 32 == 0)
                a.h_scales[mx4_scale_at(row, k, H)] = 0;
        }
        return;
    }
    // the row's own values are on their way before the first sum (of four pieces a
    // thread y alone); weights, which all rows share, are loaded where they are
    // needed: held in registers over the sums they left half as many waves, 4096 x
    // 4864 in 77 us against 48
    constexpr bool EARLY = C <= 2;
    Raw y[C], residual[C], gate[C];
    const auto load_rest = [&] {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int at = 8 * (tid + i * T);
            if (a.residual)
                residual[i] = load8(a.residual, a.r_type, row * H + at, H - at);
            if (a.gate_form & 1)  // 1: a gate a channel, 3: one a value
                gate[i] = load8(a.gate, a.gate_type, a.gate_form == 1 ? at : row * H + at, H - at);
        }
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = 8 * (tid + i * T);
        y[i] = load8(a.y, a.y_type, row * H + at, H - at);
    }
    if constexpr (EARLY)
        load_rest();
    Raw row_gate_bits = {};
    if (a.gate_form == 2)
        row_gate_bits = load8(a.gate, a.gate_type, row, 1);
    const bool post = a.post.kind, pre = a.pre.kind && a.h;
    float v[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i)
        values8(y[i], a.y_type, v[i]);
    if (post) {
        normalize<T, C>(v, a.post.kind, a.post.eps, H, part[0]);
        affine<T, C>(v, a.post, H);
    }
    if constexpr (!EARLY)
        load_rest();
    float row_gate = a.scale;
    if (a.gate_form == 2) {
        float g[8];
        values8(row_gate_bits, a.gate_type, g);
        row_gate *= g[0];
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int at = 8 * (tid + i * T);
        float f[8], g[8];
        if (a.residual) {
            values8(residual[i], a.r_type, f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = 0.f;
        }
        if (a.gate_form & 1) {
            values8(gate[i], a.gate_type, g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                g[e] *= row_gate;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                g[e] = row_gate;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = at + e < H ? __builtin_fmaf(g[e], v[i][e], f[e]) : 0.f;
        if (a.r && at < H)
            store8(a.r, a.r_type, row * H + at, H - at, v[i]);
    }
    if (!a.h)
        return;
    if (pre) {
        normalize<T, C>(v, a.pre.kind, a.pre.eps, H, part[1]);
        affine<T, C>(v, a.pre, H);
    }
    if (!a.h_scales) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int at = 8 * (tid + i * T);
            if (at < H)
                store8(a.h, a.h_type, row * H + at, H - at, v[i]);
        }
        return;
    }
    // the packed form: a block is a quad of lanes (H is a multiple of 32)
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int k = 8 * (tid + i * T);
        u32x4 bits[2];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            bits[e / 4][e % 4] = __builtin_bit_cast(uint32_t, v[i][e]);
        const uint32_t byte = scale_byte(top_of_quad(top8<2>(bits)));
        if (k < H) {
            *(uint32_t *)((uint8_t *)a.h + mx4_code_at(row, k, H)) = codes8<2>(bits, byte);
            if (k % 32 == 0)
                a.h_scales[mx4_scale_at(row, k, H)] = (uint8_t)byte;
        }
    }
    for (int k = H + 8 * tid; k < mx4_groups(H) * 512; k += 8 * T) {
        if (k < mx4_steps(H) * 128)
            *(uint32_t *)((uint8_t *)a.h + mx4_code_at(row, k, H)) = 0;
        if (k % 32 == 0)
            a.h_scales[mx4_scale_at(row, k, H)] = 0;
    }
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t stream)
{
    const int pieces = (a.H + 7) / 8, waves = (pieces + 63) / 64;
    const dim3 grid((unsigned)(a.h_scales ? (a.M + 15) / 16 * 16 : a.M));
    const auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, stream, a); };
    // one piece a thread up to 8192 values, in whole waves
    if (waves <= 1)
        go(q4_block_norm_kernel<64, 1>, 64);
    else if (waves <= 2)
        go(q4_block_norm_kernel<128, 1>, 128);
    else if (waves <= 3)
        go(q4_block_norm_kernel<192, 1>, 192);
    else if (waves <= 4)
        go(q4_block_norm_kernel<256, 1>, 256);
    else if (waves <= 5)
        go(q4_block_norm_kernel<320, 1>, 320);
    else if (waves <= 6)
        go(q4_block_norm_kernel<384, 1>, 384);
    else if (waves <= 7)
        go(q4_block_norm_kernel<448, 1>, 448);
    else if (waves <= 8)
        go(q4_block_norm_kernel<512, 1>, 512);
    else if (waves <= 10)
        go(q4_block_norm_kernel<640, 1>, 640);
    else if (waves <= 12)
        go(q4_block_norm_kernel<768, 1>, 768);
    else if (waves <= 16)
        go(q4_block_norm_kernel<1024, 1>, 1024);
    else if (waves <= 32)
        go(q4_block_norm_kernel<1024, 2>, 1024);
    else
        go(q4_block_norm_kernel<1024, 4>, 1024);
    return hipGetLastError();
}

}  // namespace q4
