// q4_moe.hip -- a mixture-of-experts layer with 4-bit experts for gfx950
// (MI355X), at the row counts of decode:
//
//     l[m][e] = sum_k x[m][k] r[e][k] + b[e]          the router's logits
//     ids, w  = the topk largest of softmax(l[m])      (lowest index first)
//     [g | u] = x[m] . dequant(W13[e])^T               for e = ids[m][j]
//     h       = g / (1 + exp(-g)) u
//     y[m]    = sum_j w[m][j] (h . dequant(W2[e])^T)   in the order of j
//
// Row invariance, as everywhere in this library: a row's bits depend on that
// row, its experts and their weights, not on the other rows.  Both products
// use the segments and the tree of q4_plan.hpp over blocks of 32.
//
// Operands.  The matrix cores take the codes as exact binary16 q - 8
// (Dequant<false>).  bfloat16 x becomes binary16 after a power of two for
// each row that puts its largest value in [2^14, 2^15): exact for every value
// down to 2^-31 of the largest.  A row is wide where that is not enough for a
// block of 32 whose largest value is below 2^-12 of the row's: then each block
// gets a further power of two that puts its own largest there.  So a value is
// exact down to 2^-19 of its block's largest and off by at most 2^-27 of it
// below (or 2^-164 of the row's, in blocks below 2^-125 of that), whatever the
// weights of the row's largest values are.  h is kept as two binary16 numbers
// (the value and what its rounding left) after a power of two for each 32
// values, 22 bits or more of each block's largest.  All sums are binary32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "q4_device.hpp"
#include "q4_launch.hpp"
#include "q4_moe_plan.hpp"

namespace q4 {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kSlots = 1024;   // (row, choice) pairs one launch handles
constexpr int kExperts = 1024;  // most experts

// ---------------------------------------------------------------- router
// Sums in binary64 (v_mfma_f64_16x16x4): the choice compares neighbouring
// logits, and 32-bit sums would let their order decide it.  The order is a
// function of K alone: chains of 64 k, four of them added in order to a part
// of 256 k, the parts added in order.
// Element kinds: 0 binary16, 1 bfloat16, 2 binary32.  Eight values of a row.
template <int KIND>
struct Eight {
    u32x4 v[KIND == 2 ? 2 : 1];
    __device__ __forceinline__ void load(const void *row, size_t k)
    {
        const u32x4 *p = (const u32x4 *)((const uint8_t *)row + k * (KIND == 2 ? 4 : 2));
        v[0] = p[0];
        if constexpr (KIND == 2)
            v[1] = p[1];
    }
    __device__ __forceinline__ double at(int i) const
    {
        if constexpr (KIND == 2) {
            const uint32_t bits = v[i / 4][i % 4];  // (a value: the cast of a vector's element in place reads element 0)
            return (double)__builtin_bit_cast(float, bits);
        } else {
            const uint32_t h = v[0][i / 2] >> (16 * (i & 1)) & 0xFFFFu;
            if constexpr (KIND == 1)
                return (double)__builtin_bit_cast(float, h << 16);
            else
                return (double)half_bits_to_float(h);
        }
    }
};

// The chain of the 64 k from k0 on (short at the end of the row): lane (g, c)
// holds expert c's (A) and row c's (B) values k = 32 s + 8 g + i of step i.
template <int XK, int RK>
__device__ __forceinline__ f64x4 logit_chain(const uint16_t *xr, const uint8_t *rr, int k0, int K, int g)
{
    f64x4 acc = {0, 0, 0, 0};
    Eight<XK> a[2];
    Eight<RK> b[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
        if (k0 + 32 * s < K) {
            a[s].load(xr, k0 + 32 * s + 8 * g);
            b[s].load(rr, k0 + 32 * s + 8 * g);
        }
#pragma unroll
    for (int s = 0; s < 2; ++s)
        if (k0 + 32 * s < K) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(b[s].at(i), a[s].at(i), acc, 0, 0, 0);
        }
    return acc;
}

// ------------------------------------------------------ x as binary16
// Exponent shift that puts a largest magnitude `top` in [2^14, 2^15), or 0 for
// zeros.
__device__ __forceinline__ int lift_of(float top)
{
    return top > 0.f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
}

// Eight bfloat16 values times 2^lift, as binary16.
__device__ __forceinline__ u32x4 lifted(u32x4 v, int lift)
{
    u32x4 out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __builtin_ldexpf(__builtin_bit_cast(float, v[i] << 16), lift);
        const float hi = __builtin_ldexpf(__builtin_bit_cast(float, v[i] & 0xFFFF0000u), lift);
        out[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
    }
    return out;
}

// The largest finite magnitude of eight bfloat16 values, with `top`.
__device__ __forceinline__ float largest(u32x4 v, float top)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __builtin_fabsf(__builtin_bit_cast(float, v[i] << 16));
        const float hi = __builtin_fabsf(__builtin_bit_cast(float, v[i] & 0xFFFF0000u));
        top = lo < __builtin_inff() ? __builtin_fmaxf(top, lo) : top;
        top = hi < __builtin_inff() ? __builtin_fmaxf(top, hi) : top;
    }
    return top;
}

// The smallest magnitude of eight bfloat16 values that is not zero, less one
// (in both halves, as bits), with `low`.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 smallest(u32x4 v, u16x2 low)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        low = __builtin_elementwise_min(low, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu) - (u16x2)(1));
    return low;
}
// Whether one of them, times 2^lift, may lie below 2^-17, from where on a
// bfloat16 number's eight bits do not fit a binary16's steps of 2^-24.
__device__ __forceinline__ bool below(u16x2 low, int lift)
{
    const uint32_t least = __builtin_bit_cast(uint32_t, __builtin_ldexpf(1.f, -17 - lift)) >> 16;
    return low.x + 1u < least || low.y + 1u < least;
}

// bfloat16 x as binary16: the rows' powers of two, which rows are wide, and
// the further powers of two of their blocks (negative: as the products take them
// back; 0 in rows that are not wide).
struct Lifted {
    uint16_t *x16;
    int *lift, *wide;
    int8_t *shift;  // [row][quads_of(K)][4]
};

__host__ __device__ inline int quads_of(int K) { return (K / 32 + 3) / 4; }

// 2^-12: hidden states with outliers of some thousand times the other values
// meet it rarely, and the bound stays below a binary32 step of the largest.
constexpr int kSpread = 12;

// Whether a row needs its blocks' own powers of two, and those: by one wave,
// four lanes a block (K % 32 = 0 keeps them together).  A further power of two
// is at most 2^125: a block scale times 2^-125 is exact (a multiple of 2^-149).
__device__ __forceinline__ bool lift_blocks(const uint16_t *x, uint16_t *x16, int8_t *shift, int up, int K)
{
    const int lane = threadIdx.x & 63;
    auto more_of = [&](u32x4 b) {
        float t = largest(b, 0.f);
        t = __builtin_fmaxf(t, __shfl_xor(t, 1));
        t = __builtin_fmaxf(t, __shfl_xor(t, 2));
        return t > 0.f ? min(lift_of(t) - up, 125) : 0;
    };
    bool need = false;
    for (int k = 8 * lane; k < K; k += 512) {
        const u32x4 b = *(const u32x4 *)(x + k);
        need |= more_of(b) > kSpread && below(smallest(b, (u16x2)(0xFFFF)), up);
    }
    if (!__any(need))
        return false;
    for (int k = 8 * lane; k < K; k += 512) {
        const u32x4 b = *(const u32x4 *)(x + k);
        const int more = more_of(b);
        *(u32x4 *)(x16 + k) = lifted(b, up + more);
        if ((lane & 3) == 0)
            shift[k / 32] = (int8_t)-more;
    }
    return true;
}

// Row m of bfloat16 x by one wave.
__device__ __forceinline__ void lift_row(const uint16_t *x_, const Lifted &to, size_t m, int K)
{
    const int lane = threadIdx.x & 63;
    constexpr int HELD = 4;  // rows up to 2048 long are read once
    const uint16_t *x = x_ + m * K;
    uint16_t *x16 = to.x16 + m * K;
    u32x4 v[HELD];
    float top = 0.f;
    u16x2 low = (u16x2)(0xFFFF);
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (8 * (lane + 64 * i) < K)
            v[i] = *(const u32x4 *)(x + 8 * (lane + 64 * i));
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (8 * (lane + 64 * i) < K) {
            top = largest(v[i], top);
            low = smallest(v[i], low);
        }
    for (int k = 8 * (lane + 64 * HELD); k < K; k += 512) {
        const u32x4 b = *(const u32x4 *)(x + k);
        top = largest(b, top);
        low = smallest(b, low);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        top = __builtin_fmaxf(top, __shfl_xor(top, d));
    const int up = lift_of(top);
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (8 * (lane + 64 * i) < K)
            *(u32x4 *)(x16 + 8 * (lane + 64 * i)) = lifted(v[i], up);
    for (int k = 8 * (lane + 64 * HELD); k < K; k += 512)
        *(u32x4 *)(x16 + k) = lifted(*(const u32x4 *)(x + k), up);
    const bool wide = __any(below(low, up)) && lift_blocks(x, x16, to.shift + m * 4 * quads_of(K), up, K);
    if (!wide)
        for (int q = lane; q < quads_of(K); q += 64)
            ((uint32_t *)to.shift)[m * quads_of(K) + q] = 0;
    if (lane == 0) {
        to.lift[m] = up;
        to.wide[m] = wide;
    }
}

__global__ __launch_bounds__(256) void q4_moe_lift_kernel(const uint16_t *__restrict__ x, Lifted to, int M, int K)
{
    const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m < M)
        lift_row(x, to, m, K);
}

// Few rows: grid = (16-expert tiles, 16-row tiles, parts), a wave a chain; the
// reader adds the parts.  One more z takes the rows to binary16 (to.x16 given).
// One row of 64 experts over 2048: 3.3 us, launch and latency (a workgroup per
// 16 experts over all of K, its waves on every 16th chunk, took 7).  201 rows of
// 127 experts over 3584, binary32 router: 9 us, conversions to binary64 and
// the products.
template <int XK, int RK>
__global__ __launch_bounds__(256) void q4_moe_logits_kernel(const uint16_t *__restrict__ x,
                                                            const void *__restrict__ router,
                                                            double *__restrict__ parts, Lifted to, int M, int E,
                                                            int K)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int part = blockIdx.z;
    if (part * kPart >= K) {
        const int all = gridDim.x * gridDim.y * 4;
        for (int m = (blockIdx.y * gridDim.x + blockIdx.x) * 4 + wave; m < M; m += all)
            lift_row(x, to, m, K);
        return;
    }
    const int e = min((int)blockIdx.x * 16 + c, E - 1), m = min((int)blockIdx.y * 16 + c, M - 1);
    const f64x4 acc = logit_chain<XK, RK>(x + (size_t)m * K,
                                          (const uint8_t *)router + (size_t)e * K * (RK == 2 ? 4 : 2),
                                          part * kPart + 64 * wave, K, g);
    __shared__ double chain[4][4][64];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        chain[wave][i][lane] = acc[i];
    __syncthreads();
    const double s = ((chain[0][wave][lane] + chain[1][wave][lane]) + chain[2][wave][lane]) + chain[3][wave][lane];
    // component i of lane (g, c): expert 4 i + g of the tile, row c
    const int oe = blockIdx.x * 16 + 4 * wave + g, om = blockIdx.y * 16 + c;
    if (oe < E && om < M)
        parts[((size_t)part * M + om) * E + oe] = s;
}

// Many rows: a wave owns 16 experts by 16 rows over all of K, the same sums.
template <int XK, int RK>
__global__ __launch_bounds__(256) void q4_moe_logits_rows_kernel(const uint16_t *__restrict__ x,
                                                                 const void *__restrict__ router,
                                                                 double *__restrict__ logits, int M, int E, int K)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int et = blockIdx.x, mt = blockIdx.y * 4 + wave;
    if (mt * 16 >= M)
        return;
    const int e = min(et * 16 + c, E - 1), m = min(mt * 16 + c, M - 1);
    const uint16_t *xr = x + (size_t)m * K;
    const uint8_t *rr = (const uint8_t *)router + (size_t)e * K * (RK == 2 ? 4 : 2);
    f64x4 sum = {0, 0, 0, 0};
    for (int k = 0; k < K; k += kPart) {
        f64x4 p = logit_chain<XK, RK>(xr, rr, k, K, g);
#pragma unroll
        for (int w = 1; w < 4; ++w)
            p += logit_chain<XK, RK>(xr, rr, k + 64 * w, K, g);
        sum = k ? sum + p : p;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int oe = et * 16 + 4 * i + g, om = mt * 16 + c;
        if (oe < E && om < M)
            logits[(size_t)om * E + oe] = sum[i];
    }
}

// A logit as an integer of the same order, NaN above everything.
__device__ __forceinline__ uint64_t order_key(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    if (v != v)
        return ~0ull;
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double key_value(uint64_t k)
{
    if (k == ~0ull)
        return __builtin_nan("");
    return __builtin_bit_cast(double, k >> 63 ? k ^ (1ull << 63) : ~k);
}

// What a workgroup needs to choose its rows' experts from the logits' parts.
struct Choice {
    const double *parts;  // [count][M][E]
    const float *bias;    // or null
    int count, M, E, topk, renormalize;
};

// Rows m0 .. m0 + rows - 1 by a workgroup: every expert's rank in its row is the
// number of experts before it (a larger logit, or an equal one at a lower
// index), spread over as many threads as there are; the first topk ranks are
// the choice.  keys: rows E numbers of LDS; chosen: rows topk.  ids goes to
// LDS (ids_out + row topk) and, as the weights, to memory where asked.
template <typename ID>
__device__ __forceinline__ void choose_rows(const Choice &ch, int m0, int rows, uint64_t *keys, double *chosen,
                                            ID *ids_lds, int *ids, float *weights, bool out)
{
    const int tid = threadIdx.x, T = blockDim.x, E = ch.E, topk = ch.topk;
    const int pairs = rows * E;
    for (int p = tid; p < pairs; p += T) {
        const double *at = ch.parts + (size_t)m0 * E + p;
        const size_t step = (size_t)ch.M * E;
        double l = 0.0;  // (0 + the first part: that part, but for the sign of a zero)
        for (int i0 = 0; i0 < ch.count; i0 += 8) {
            double v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = i0 + i < ch.count ? at[(i0 + i) * step] : 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                l += v[i];
        }
        if (ch.bias)
            l += (double)ch.bias[p % E];
        keys[p] = order_key(l);
    }
    __syncthreads();
    int share = 1;  // threads a pair
    while (2 * share * pairs <= T && share < 64)
        share *= 2;
    const int at = tid % share;
    for (int p = tid / share; p < pairs; p += T / share) {
        const int row = p / E, e = p - row * E;
        const uint64_t key = keys[p], *k = keys + row * E;
        int rank = 0;
        for (int f0 = at; f0 < E; f0 += 8 * share) {  // (eight at a time: one wait for LDS; 0 is below every key)
            uint64_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = f0 + i * share < E ? k[f0 + i * share] : 0ull;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                rank += (o[i] > key) | ((o[i] == key) & (f0 + i * share < e));
        }
        for (int d = 1; d < share; d *= 2)
            rank += __shfl_xor(rank, d);
        if (at == 0 && rank < topk) {
            const double v = key_value(key);
            chosen[row * topk + rank] = v;
            const int id = v == -__builtin_inf() ? -1 : e;
            if (ids_lds)
                ids_lds[row * topk + rank] = (ID)id;
            if (out)
                ids[(size_t)(m0 + row) * topk + rank] = id;
        }
    }
    __syncthreads();
    if (!out)
        return;
    // softmax over all experts, or over the chosen ones: a wave a row
    const int lane = tid & 63;
    for (int row = tid >> 6; row < rows; row += T >> 6) {
        const double *c = chosen + row * topk;
        const double top = c[0];
        float sum = 0.f;
        const int n = ch.renormalize ? topk : E;
        for (int i = lane; i < n; i += 64) {
            const double v = ch.renormalize ? c[i] : key_value(keys[row * E + i]);
            sum += v == -__builtin_inf() ? 0.f : __builtin_expf((float)(v - top));
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2)
            sum += __shfl_xor(sum, d);
        for (int i = lane; i < topk; i += 64) {
            const double v = c[i];
            weights[(size_t)(m0 + row) * topk + i] =
                v == -__builtin_inf() ? 0.f : __builtin_expf((float)(v - top)) / sum;
        }
    }
}

// A workgroup a row; with to.x16, the last wave takes the row to binary16 first.
// 3.2 us at one row of 64 experts, 5.5 at 201 rows of 127: latency.
__global__ __launch_bounds__(512) void q4_moe_select_kernel(Choice ch, int *__restrict__ ids,
                                                            float *__restrict__ weights,
                                                            const uint16_t *__restrict__ x, Lifted to, int K)
{
    extern __shared__ double row[];  // E keys, then topk chosen logits
    const size_t m = blockIdx.x;
    if (to.x16 && threadIdx.x >= 448)
        lift_row(x, to, m, K);
    choose_rows<int>(ch, (int)m, 1, (uint64_t *)row, row + ch.E, nullptr, ids, weights, true);
}

// -------------------------------------------------------- expert products
// Row slots: batch row i of a group of 4 R rows sits, for block j of a quad,
// in the operand and A row slot that `Slots<R>` gives; its value of block j
// then lands in component comp(j, r) of lane group i % 4 with r = i / 4 (the
// layout of gemv_quad_slots and gemv_quad_slots2).
template <int R>
struct Slots;
template <>
struct Slots<1> {
    static __device__ __forceinline__ int row(int c) { return c >> 2; }
    static __device__ __forceinline__ int block(int, int c) { return c & 3; }
    static __device__ __forceinline__ constexpr int operand(int) { return 0; }
    static __device__ __forceinline__ constexpr int comp(int j, int) { return j; }
};
template <>
struct Slots<2> {
    static __device__ __forceinline__ int row(int c) { return (c >> 2) + 4 * (c & 1); }
    static __device__ __forceinline__ int block(int o, int c) { return 2 * o + ((c & 3) >> 1); }
    static __device__ __forceinline__ constexpr int operand(int j) { return j >> 1; }
    static __device__ __forceinline__ constexpr int comp(int j, int r) { return 2 * (j & 1) + r; }
};
template <>
struct Slots<4> {
    static __device__ __forceinline__ int row(int c) { return (c >> 2) + 4 * (c & 3); }
    static __device__ __forceinline__ int block(int o, int) { return o; }
    static __device__ __forceinline__ constexpr int operand(int j) { return j; }
    static __device__ __forceinline__ constexpr int comp(int, int r) { return r; }
};

// Buffer loads: a wave-uniform base with the range of what may be read, a
// lane's own 32-bit offset and a uniform one, so that a stream costs one
// register a lane.  A lane's offset of kNowhere is past every range (they stay
// below 2^29 bytes): it reads zero.  The uniform offset itself stays within the
// range, so that nothing hangs on how the check takes one past it.
constexpr uint32_t kNowhere = 1u << 31;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, size_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t at, uint32_t uniform)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at, uniform, 0));
}
// Codes and scales are read once a call: the non-temporal hint, as in the
// 4-bit product's kernels.
__device__ __forceinline__ u32x4 load_codes(__amdgpu_buffer_rsrc_t b, uint32_t at, int q)
{
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, at, 1024 * q, 2));
}
__device__ __forceinline__ u32x2 load_scales(__amdgpu_buffer_rsrc_t b, uint32_t at, int q)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, at, 128 * q, 2));
}
// A tile of 16 columns: its codes and scales over all of K.
struct Tile {
    __amdgpu_buffer_rsrc_t w, s;
    Tile() = default;
    __device__ __forceinline__ Tile(const uint8_t *wq, const uint16_t *scales, size_t tile, int G)
        : w(buffer_of(wq + tile * G * 1024, (size_t)G * 1024)), s(buffer_of(scales + tile * G * 64, (size_t)G * 128))
    {
    }
};
__device__ __forceinline__ float quad_scale(u32x2 s, int j)
{
    return half_bits_to_float((j < 2 ? s.x : s.y) >> (16 * (j & 1)) & 0xFFFFu);
}

__device__ __forceinline__ f32x4 dot16(u32x4 a, u32x4 b, f32x4 c) { return blockdot_acc<false>(a, b, c); }

__device__ __forceinline__ int slot_expert(int id, int E) { return id >= 0 && id < E ? id : -1; }

// The expert of a workgroup and its slots.
struct Found {
    uint16_t list[kSlots];
    int16_t who[kSlots];  // the slots' experts where this kernel chose them
};

// Workgroup `nth` of a grid of min(n, E): with as many slots as experts or
// more, it is expert nth's; else it is slot nth's expert's, if that is the
// expert's first slot.  Every wave finds its slots alone (a compare and a
// ballot for 64 slots), without a barrier, all writing the same list, and
// `start` sends for its weights as soon as the expert is known.  -> how many
// slots, 0 for a workgroup without work.
template <typename START>
__device__ __forceinline__ int find_expert(Found &f, int n, const int *ids, bool known, int E, int nth, START start)
{
    const int lane = threadIdx.x & 63;
    auto who = [&](int s) { return known ? (int)f.who[s] : slot_expert(ids[s], E); };
    const bool by_slot = n < E;
    int e = nth;
    if (by_slot) {
        e = __builtin_amdgcn_readfirstlane(who(nth));
        if (e < 0)
            return 0;
    }
    int count = 0;
    bool started = false;
    for (int s0 = 0; s0 < n; s0 += 256) {
        int id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            id[i] = s0 + 64 * i + lane < n ? who(s0 + 64 * i + lane) : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t mask = __ballot(id[i] == e);
            if (!mask)
                continue;
            if (!started) {
                if (by_slot && s0 + 64 * i + __builtin_ctzll(mask) != nth)
                    return 0;
                start(e);
                started = true;
            }
            if (mask >> lane & 1)
                f.list[count + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)(s0 + 64 * i + lane);
            count += __popcll(mask);
        }
    }
    __threadfence_block();
    return count;
}

// What a workgroup multiplies: four tiles of 16 columns of one expert's weight
// (the quads of K are the waves' runs of L segments).
struct FourTiles {
    Tile t0, t1, t2, t3;
};
struct Weights {
    u32x4 codes[4];
    u32x2 scales[4];
    // Quad q of the tiles, or nothing from quad qb on: always the same loads, so
    // that the wait for the quad before never has to be a wait for them too.
    __device__ __forceinline__ void load(const FourTiles &f, int q, int qb)
    {
        const uint32_t lane = threadIdx.x & 63;
        const uint32_t w_at = q < qb ? 16 * lane : kNowhere, s_at = q < qb ? 8 * (lane & 15) : kNowhere;
        q = min(q, qb - 1);
        codes[0] = load_codes(f.t0.w, w_at, q);
        codes[1] = load_codes(f.t1.w, w_at, q);
        codes[2] = load_codes(f.t2.w, w_at, q);
        codes[3] = load_codes(f.t3.w, w_at, q);
        scales[0] = load_scales(f.t0.s, s_at, q);
        scales[1] = load_scales(f.t1.s, s_at, q);
        scales[2] = load_scales(f.t2.s, s_at, q);
        scales[3] = load_scales(f.t3.s, s_at, q);
    }
};

// Keeps loads ahead of what follows them (no instructions).
__device__ __forceinline__ void issue_fence()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// x as the gate/up kernel takes it: binary16, with the rows' powers of two and
// wide rows where it was bfloat16 (else null).
struct UpIn {
    const uint16_t *x;
    const int *lift, *wide;
    const int8_t *shift;
    int M, H;
};

// The rows' operands of one quad; where WIDE, with the further powers of two of
// the rows whose values the lane group accumulates (2^0 in rows that are not
// wide, and the same bits).  row(i): the batch row of row i of the group.
template <int R, bool WIDE>
struct RowsX {
    u32x4 x[R];
    uint32_t shift[WIDE ? R : 1];
    struct In {
        __amdgpu_buffer_rsrc_t x, shift;
        uint32_t at, shift_at[WIDE ? R : 1];
        int nb, last;
    };
    template <typename ROW>
    static __device__ __forceinline__ In in(const UpIn &u, ROW row, int rows, int nb)
    {
        const int lane = threadIdx.x & 63, g = lane >> 4, i = Slots<R>::row(lane & 15);
        In in;
        in.x = buffer_of(u.x, (size_t)u.M * u.H * 2);
        in.at = i < rows ? (uint32_t)row(i) * 2u * u.H + 16 * g : kNowhere;
        if constexpr (WIDE) {
            const int pitch = 4 * quads_of(u.H);
            in.shift = buffer_of(u.shift, (size_t)u.M * pitch);
#pragma unroll
            for (int r = 0; r < R; ++r)
                in.shift_at[r] = 4 * r + g < rows ? (uint32_t)row(4 * r + g) * pitch : kNowhere;
        }
        in.nb = nb;
        in.last = (nb - 1) / 4;
        return in;
    }
    __device__ __forceinline__ void load(const In &in, int q)
    {
        const int c = threadIdx.x & 15, to = min(q, in.last);
#pragma unroll
        for (int o = 0; o < R; ++o) {  // (blocks past the end of a short last quad: zero)
            const int b = Slots<R>::block(o, c);
            x[o] = load16(in.x, 4 * q + b < in.nb ? in.at + 64 * b : kNowhere, 256 * to);
        }
        if constexpr (WIDE)
#pragma unroll
            for (int r = 0; r < R; ++r)
                shift[r] = __builtin_amdgcn_raw_buffer_load_b32(in.shift, in.shift_at[r], 4 * to, 0);
    }
    __device__ __forceinline__ f32x4 dot(int j, u32x4 b) const { return blockdot<false>(x[Slots<R>::operand(j)], b); }
    __device__ __forceinline__ float scale(float d, int r, int j) const
    {
        if constexpr (WIDE)
            return __builtin_ldexpf(d, (int)(int8_t)(shift[r] >> (8 * j)));
        else
            return d;
    }
};

// h as the gate/up kernel leaves it.
struct DownIn {
    const uint16_t *hi, *lo;
    const int *shift;
    int n, I, shifts;  // slots, values and powers of two of a slot
};

// A row's operands of h for one quad: both halves, and the powers of two of the
// rows whose values the lane group accumulates.
template <int R>
struct RowsH {
    u32x4 hi[R], lo[R], shift[R];
    struct In {
        __amdgpu_buffer_rsrc_t hi, lo, shift;
        uint32_t at, shift_at[R];
        int nb, last;
    };
    static __device__ __forceinline__ In in(const DownIn &h, const uint16_t *list, int rows, int nb)
    {
        const int lane = threadIdx.x & 63, g = lane >> 4, row = Slots<R>::row(lane & 15);
        In i;
        i.hi = buffer_of(h.hi, (size_t)h.n * h.I * 2);
        i.lo = buffer_of(h.lo, (size_t)h.n * h.I * 2);
        i.shift = buffer_of(h.shift, (size_t)h.n * h.shifts * 4);
        i.at = row < rows ? (uint32_t)list[row] * 2u * h.I + 16 * g : kNowhere;
#pragma unroll
        for (int r = 0; r < R; ++r)
            i.shift_at[r] = 4 * r + g < rows ? (uint32_t)list[4 * r + g] * 4u * h.shifts : kNowhere;
        i.nb = nb;
        i.last = (nb - 1) / 4;
        return i;
    }
    __device__ __forceinline__ void load(const In &in, int q)
    {
        const int c = threadIdx.x & 15, to = min(q, in.last);
#pragma unroll
        for (int o = 0; o < R; ++o) {  // (blocks past the end of a short last quad: zero)
            const int b = Slots<R>::block(o, c);
            const uint32_t at = 4 * q + b < in.nb ? in.at + 64 * b : kNowhere;
            hi[o] = load16(in.hi, at, 256 * to);
            lo[o] = load16(in.lo, at, 256 * to);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            shift[r] = load16(in.shift, in.shift_at[r], 16 * to);
    }
    __device__ __forceinline__ f32x4 dot(int j, u32x4 b) const
    {
        return dot16(hi[Slots<R>::operand(j)], b, blockdot<false>(lo[Slots<R>::operand(j)], b));
    }
    __device__ __forceinline__ float scale(float d, int r, int j) const
    {
        return __builtin_ldexpf(d, (int)shift[r][j]);
    }
};

// The products of up to 4 R rows (operands ROWS) with the wave's run of L
// segments of four tiles, a quad of both loaded ahead (the first quad's
// weights by the caller).  The run's part of the tree waits in the wave's own
// LDS, stack [level][tile][r][lane] (levels that the trailing one-bits of a
// segment's number name are merged, left operand first), and ends in level 0.
template <int R, typename ROWS>
__device__ __forceinline__ void multiply_run(const FourTiles &tiles, Weights &first, const typename ROWS::In &in, int sa,
                                             int L, const Plan &plan, float *stack)
{
    const int lane = threadIdx.x & 63;
    const Dequant<false> dq;
    const int qa = (sa * plan.G) >> plan.log2S, qb = ((sa + L) * plan.G) >> plan.log2S;
    float p[4][R];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r)
            p[t][r] = 0.f;
    int seg = 0, end = ((sa + 1) * plan.G) >> plan.log2S;
    auto multiply = [&](const Weights &w, const ROWS &x, int q) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4 D[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                D[j] = x.dot(j, dq(w.codes[t][j]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = quad_scale(w.scales[t], j);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    p[t][r] = __builtin_fmaf(x.scale(d, r, j), D[j][Slots<R>::comp(j, r)], p[t][r]);
            }
        }
        if (q + 1 == end) {  // a segment ends
            int level = 0;
            for (; seg >> level & 1; ++level)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        p[t][r] = stack[((level * 4 + t) * R + r) * 64 + lane] + p[t][r];
            if (seg == L - 1)
                level = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    stack[((level * 4 + t) * R + r) * 64 + lane] = p[t][r];
                    p[t][r] = 0.f;
                }
            ++seg;
            end = ((sa + seg + 1) * plan.G) >> plan.log2S;
        }
    };
    Weights second;
    ROWS xa, xb;
    xa.load(in, qa);
    for (int q = qa; q < qb; q += 2) {
        second.load(tiles, q + 1, qb);
        xb.load(in, q + 1);
        issue_fence();
        multiply(first, xa, q);
        first.load(tiles, q + 2, qb);
        xa.load(in, q + 2);
        issue_fence();
        if (q + 1 < qb)
            multiply(second, xb, q + 1);
    }
}

// What the join of a group's sums needs: the waves' roots, `step` numbers apart.
struct Roots {
    const float *part;
    int waves, step;
};

// Output (tile, row i of a group, column c): the top of the tree.
template <int R>
__device__ __forceinline__ float join_roots(const Roots &at, int tile, int i, int c)
{
    const float *p = at.part + (tile * R + (i >> 2)) * 64 + (i & 3) * 16 + c;
    if (at.waves == 1)
        return p[0];
    float v[8];
#pragma unroll
    for (int w = 0; w < 8; ++w)
        v[w] = w < at.waves ? p[w * at.step] : 0.f;
    return tree_sum<8>(v, at.waves);
}

// gate and up: a unit is two tiles of gate and two of up, so that it ends with
// 32 values of h, one block of the down product.
template <bool BF16>
struct Up {
    UpIn x;
    uint16_t *hi, *lo;
    int *shift;
    int topk, I, shifts;

    // waves of a compute unit's quarter that the registers are to hold
    static constexpr int waves(int RM) { return RM == 1 ? 4 : 3; }
    template <int R, bool WIDE>
    using Rows = RowsX<R, WIDE>;
    // Groups of 4 and 8 rows carry the powers of two of bfloat16's blocks always
    // (a load and four operations a tile and quad: 0.4 to 1.3 us a layer), groups
    // of 16 have no registers for them (27 spilled): a batch with a wide row goes 4
    // rows at a time there (64 rows of 64 experts 3584 x 1792: 167 -> 238 us).
    static constexpr bool always(int RM) { return BF16 && RM <= 2; }
    static constexpr bool asks(int RM) { return BF16 && RM > 2; }
    // what a lane knows of the wide rows of the batch: loaded first, used after
    // the weights are on their way
    __device__ __forceinline__ int wide() const
    {
        int m = threadIdx.x & 63, any = m < x.M ? x.wide[m] : 0;
        if (x.M > 64)
            for (m += 64; m < x.M; m += 64)
                any |= x.wide[m];
        return any;
    }
    __host__ __device__ int units() const { return I / 32; }
    __device__ __forceinline__ FourTiles tiles(const uint8_t *wq, const uint16_t *scales, int e, int unit, int G) const
    {
        const size_t gate = (size_t)e * (2 * I / 16) + 2 * unit, up = gate + I / 16;
        return FourTiles{Tile(wq, scales, gate, G), Tile(wq, scales, gate + 1, G), Tile(wq, scales, up, G),
                         Tile(wq, scales, up + 1, G)};
    }
    template <int R, bool WIDE>
    __device__ __forceinline__ typename RowsX<R, WIDE>::In in(const uint16_t *list, int rows, int nb) const
    {
        return RowsX<R, WIDE>::in(x, [&](int i) { return list[i] / topk; }, rows, nb);
    }
    // (loaded before the products, used after them)
    __device__ __forceinline__ int before(const uint16_t *list, int rows) const
    {
        return BF16 && (int)threadIdx.x < rows ? -x.lift[list[threadIdx.x] / topk] : 0;
    }
    // 32 lanes a row: the trees, the activation, the block's power of two
    template <int R>
    __device__ __forceinline__ void after(const Roots &roots, const int *back, const uint16_t *list, int rows,
                                          int unit) const
    {
        for (int o = threadIdx.x; o < rows * 32; o += blockDim.x) {
            const int i = o >> 5, col = o & 31;
            const float gate = __builtin_ldexpf(join_roots<R>(roots, col >> 4, i, col & 15), back[i]);
            const float up = __builtin_ldexpf(join_roots<R>(roots, 2 + (col >> 4), i, col & 15), back[i]);
            // exp(-gate) passes the largest number from -88.8 down; there h is gate exp(gate) up within
            // 2^-115 of it, by halves of the exponential, so that no factor underflows before h does
            float h;
            if (gate < -80.f) {
                const float e = __builtin_expf(0.5f * gate);
                h = (gate * e) * (up * e);
            } else {
                h = gate / (1.f + __builtin_expf(-gate)) * up;
            }
            float top = __builtin_fabsf(h) < __builtin_inff() ? __builtin_fabsf(h) : 0.f;
#pragma unroll
            for (int d = 1; d < 32; d *= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, d));
            // (at most 2^125: a block scale times 2^-125 in the down product is exact, a
            // multiple of 2^-149, and h 2^125 one of 2^-24, as binary16 holds it)
            const int raise = min(lift_of(top), 125);
            const float v = __builtin_ldexpf(h, raise);
            const _Float16 vh = (_Float16)v;
            const float rest = v - (float)vh;
            const _Float16 vl = __builtin_fabsf(v) < __builtin_inff() ? (_Float16)rest : (_Float16)0.f;
            const size_t slot = list[i];
            const size_t k = slot * I + 32 * unit + col;
            hi[k] = __builtin_bit_cast(uint16_t, vh);
            lo[k] = __builtin_bit_cast(uint16_t, vl);
            if (col == 0)
                shift[slot * shifts + unit] = -raise;
        }
    }
};

// down: a unit is 64 columns, so that h is read once for four tiles; each (row,
// expert) pair's product goes to memory (t [slot][H]).
struct Down {
    DownIn h;
    float *t;
    int H;

    static constexpr int waves(int RM) { return RM == 1 ? 4 : RM == 2 ? 3 : 2; }
    template <int R, bool>
    using Rows = RowsH<R>;
    static constexpr bool always(int) { return false; }
    static constexpr bool asks(int) { return false; }
    __device__ __forceinline__ int wide() const { return 0; }
    __host__ __device__ int units() const { return (H + 63) / 64; }
    // (past the last column: the last tile, its values are not stored)
    __device__ __forceinline__ FourTiles tiles(const uint8_t *wq, const uint16_t *scales, int e, int unit, int G) const
    {
        const size_t base = (size_t)e * (H / 16);
        const int at = 4 * unit, last = H / 16 - 1;
        return FourTiles{Tile(wq, scales, base + at, G), Tile(wq, scales, base + min(at + 1, last), G),
                         Tile(wq, scales, base + min(at + 2, last), G), Tile(wq, scales, base + min(at + 3, last), G)};
    }
    template <int R, bool>
    __device__ __forceinline__ typename RowsH<R>::In in(const uint16_t *list, int rows, int nb) const
    {
        return RowsH<R>::in(h, list, rows, nb);
    }
    __device__ __forceinline__ int before(const uint16_t *, int) const { return 0; }
    template <int R>
    __device__ __forceinline__ void after(const Roots &roots, const int *, const uint16_t *list, int rows,
                                          int unit) const
    {
        for (int o = threadIdx.x; o < rows * 64; o += blockDim.x) {
            const int i = o >> 6, col = 64 * unit + (o & 63);
            if (col < H)
                t[(size_t)list[i] * H + col] = join_roots<R>(roots, (o & 63) >> 4, i, o & 15);
        }
    }
};

// Levels of the tree that wait within a run of L segments.
__host__ __device__ inline int tree_levels(int L)
{
    int n = 1;
    while (2 << n <= L)
        ++n;
    return n;
}

// One product of the layer.  grid = (units, min(slots, E), Z): a unit of four
// tiles of one expert a workgroup, its waves on runs of L segments of K.  An
// expert's rows go 4 RM at a time (the last ones 4, 8 or 16, by how many are
// left), group r to the workgroup z = r mod Z; the weights of the next group's
// first quad are on their way while this one's sums are joined.
// Few rows: bound by launch and memory latency (64 experts 2048 x 1024 at one
// row: gate/up with its choice 11.1 us, down 6.5 us).  Many: by the weights'
// stream and the dequantization's issue (47 VALU operations a tile and quad, half of
// the cycles) that overlap in part: 64 experts 3584 x 1792 at 64 rows, gate/up
// 94 us (4.9 TB/s), down 69 us (3.4 TB/s); without the products the layer took
// 152 of then 205 us.
template <typename OP, int RM>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(OP::waves(RM)))) void q4_moe_product_kernel(
    Choice ch, OP op, int *__restrict__ ids, float *__restrict__ weights, const uint8_t *__restrict__ wq,
    const uint16_t *__restrict__ scales, int L, Plan plan)
{
    extern __shared__ __attribute__((aligned(16))) float part[];  // [wave][level][tile][r][lane]
    __shared__ Found found;
    __shared__ int back[16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int levels = tree_levels(L);
    const int wide_lane = OP::asks(RM) ? op.wide() : 0;
    if (ch.parts) {
        uint64_t *keys = (uint64_t *)part;
        choose_rows<int16_t>(ch, 0, ch.M, keys, (double *)(keys + ch.M * ch.E), found.who, ids, weights,
                             blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
        __syncthreads();  // (the keys' room is the products' next)
    }
    const int qa = (wave * L * plan.G) >> plan.log2S, qb = ((wave + 1) * L * plan.G) >> plan.log2S;
    FourTiles tiles;
    Weights first;
    const int count = find_expert(found, ch.M * ch.topk, ids, ch.parts != nullptr, ch.E, blockIdx.y, [&](int e) {
        tiles = op.tiles(wq, scales, e, blockIdx.x, plan.G);
        first.load(tiles, qa, qb);
    });
    const bool wide = OP::asks(RM) && __any(wide_lane);
    const int most = wide ? 4 : 4 * RM, step = most * gridDim.z;
    for (int r0 = most * blockIdx.z; r0 < count; r0 += step) {
        const int left = min(count - r0, most);
        const uint16_t *list = found.list + r0;
        auto group = [&](auto r, auto w) {
            constexpr int R = decltype(r)::value;
            constexpr bool WIDE = decltype(w)::value;
            const int b = op.before(list, left);
            multiply_run<R, typename OP::template Rows<R, WIDE>>(
                tiles, first, op.template in<R, WIDE>(list, left, plan.nb), wave * L, L, plan,
                part + wave * levels * 4 * R * 64);
            if ((int)threadIdx.x < 16)
                back[threadIdx.x] = b;
            if (r0 + step < count)
                first.load(tiles, qa, qb);
            __syncthreads();
            op.template after<R>(Roots{part, waves, levels * 4 * R * 64}, back, list, left, blockIdx.x);
            if (r0 + step < count)
                __syncthreads();  // the sums are read
        };
        typedef std::integral_constant<bool, OP::always(RM)> Always;
        if (OP::asks(RM) && wide)
            group(std::integral_constant<int, 1>(), std::integral_constant<bool, OP::asks(RM)>());
        else if (RM == 1 || left <= 4)
            group(std::integral_constant<int, 1>(), Always());
        else if (RM == 2 || left <= 8)
            group(std::integral_constant<int, RM == 1 ? 1 : 2>(), Always());
        else
            group(std::integral_constant<int, RM>(), Always());
    }
}

// y[m] = sum_j weights[m][j] t[m, j], in the order of j.  grid = (256 columns,
// rows).  The choice and the products are loaded together, whether a slot has
// an expert or not (a slot without one holds no product: its values are not
// used).  One memory latency: 2 to 4 us.
__global__ __launch_bounds__(64) void q4_moe_join_kernel(const int *__restrict__ ids, const float *__restrict__ weights,
                                                         const float *__restrict__ t, float *__restrict__ y, int topk,
                                                         int E, int H, int vec)
{
    const int col = (blockIdx.x * 64 + threadIdx.x) * 4;
    const size_t m = blockIdx.y;
    if (col >= H)
        return;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < topk; j0 += 8) {
        f32x4 v[8];
        float w[8];
        int id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const size_t slot = m * topk + min(j0 + j, topk - 1);
            id[j] = ids[slot];
            w[j] = weights[slot];
            v[j] = *(const f32x4 *)(t + slot * H + col);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < topk && slot_expert(id[j], E) >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[i] = __builtin_fmaf(w[j], v[j][i], sum[i]);
            }
    }
    float *out = y + m * H + col;
    if (vec) {
        *(f32x4 *)out = sum;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = sum[i];
    }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Rows one launch handles.
int chunk_rows(int M, int topk) { return std::min(M, kSlots / topk); }

template <int XK, int RK>
void launch_logits_k(const uint16_t *x, const void *router, double *parts, const Lifted &to, int M, int E, int K,
                     hipStream_t stream)
{
    const int count = logit_parts(M, E, K);
    const unsigned et = (unsigned)((E + 15) / 16), mt = (unsigned)((M + 15) / 16);
    if (moe_by_rows(M, E, K))
        hipLaunchKernelGGL((q4_moe_logits_rows_kernel<XK, RK>), dim3(et, (mt + 3) / 4), dim3(256), 0, stream, x, router,
                           parts, M, E, K);
    else
        hipLaunchKernelGGL((q4_moe_logits_kernel<XK, RK>), dim3(et, mt, (unsigned)(count + (to.x16 ? 1 : 0))), dim3(256),
                           0, stream, x, router, parts, to, M, E, K);
}

hipError_t launch_logits(const void *x, int xk, const void *router, int rk, double *parts, const Lifted &to, int M,
                         int E, int K, hipStream_t stream)
{
    const uint16_t *xp = (const uint16_t *)x;
    if (xk == 1 && rk == 2)
        launch_logits_k<1, 2>(xp, router, parts, to, M, E, K, stream);
    else if (xk == 1)
        launch_logits_k<1, 1>(xp, router, parts, to, M, E, K, stream);
    else if (rk == 2)
        launch_logits_k<0, 2>(xp, router, parts, to, M, E, K, stream);
    else
        launch_logits_k<0, 0>(xp, router, parts, to, M, E, K, stream);
    return hipGetLastError();
}

hipError_t launch_select(const Choice &ch, int *ids, float *weights, const void *x, const Lifted &to, int K,
                         hipStream_t stream)
{
    hipLaunchKernelGGL(q4_moe_select_kernel, dim3((unsigned)ch.M), dim3(512),
                       (size_t)(ch.E + ch.topk) * sizeof(double), stream, ch, ids, weights, (const uint16_t *)x, to,
                       K);
    return hipGetLastError();
}

// Where the parts of a workspace lie; sizes of a piece of rows.
struct MoeRoom {
    uint16_t *hi, *lo;
    int *shift;
    Lifted x;  // where x is bfloat16
    float *t;
    size_t bytes;
    MoeRoom(void *base, int rows, int topk, int H, int I)
    {
        const size_t n = (size_t)rows * topk;
        uint8_t *p = (uint8_t *)base;
        size_t at = 0;
        auto take = [&](size_t b) {
            uint8_t *r = p + at;
            at += up256(b);
            return r;
        };
        hi = (uint16_t *)take(n * I * 2);
        lo = (uint16_t *)take(n * I * 2);
        shift = (int *)take(n * shifts_of(I) * 4);
        x.x16 = (uint16_t *)take((size_t)rows * H * 2);
        x.lift = (int *)take((size_t)rows * 4);
        x.wide = (int *)take((size_t)rows * 4);
        x.shift = (int8_t *)take((size_t)rows * 4 * quads_of(H));
        t = (float *)take(n * H * 4);
        bytes = at;
    }
    // What gate/up reads: binary16 x as given, or what lift_row leaves.
    UpIn in(const void *given, bool bf16, int M, int H) const
    {
        return bf16 ? UpIn{x.x16, x.lift, x.wide, x.shift, M, H}
                    : UpIn{(const uint16_t *)given, nullptr, nullptr, nullptr, M, H};
    }
    // an expert row's powers of two, padded to whole quads
    static int shifts_of(int I) { return 4 * quads_of(I); }
};

// The largest group of rows a product is built for (4 RM): by the rows an
// expert gets on average.  A group takes a weight through its dequantization
// once, a larger one costs registers: 64 experts 3584 x 1792 with 6 rows each
// in groups of at most 8 / 16 188 / 168 us, 128 experts 2048 x 768 with 4 rows
// each 96 / 98 us.  An average knows nothing of skewed routing, and the launch
// nothing of the routing at all: 64 rows with 8 of those 128 experts take 90 us
// with uniform choices (12 rows an expert at most), 127 where expert i is chosen
// in proportion to 1 / i (44 at most, 105 experts read), 160 where one expert is
// in every row; 64 rows with 6 of 64 experts 3584 x 1792 166, 179 and 174.
int row_group(int n, int E)
{
    const int rows = n / std::min(n, E);
    return rows <= 1 ? 1 : rows <= 4 ? 2 : 4;
}

template <typename OP, int RM>
hipError_t launch_product_r(const Choice &ch, const OP &op, int *ids, float *weights, const uint8_t *wq,
                            const uint16_t *scales, const Plan &plan, hipStream_t stream)
{
    const int n = ch.M * ch.topk;
    // as many workgroups for an expert's rows as it has groups of 16 on average,
    // up to four: the layer of 8 experts 2048 x 512 with 64 rows each 71 us with
    // one, 53 with four; 1024 x 1024 with 256 rows each 285, 151, without a
    // limit 238 (each reads the weights again)
    const int experts = std::min(n, ch.E), groups = RM == 4 ? std::min(n / experts / 16 + 1, 4) : 1;
    const dim3 grid((unsigned)op.units(), (unsigned)experts, (unsigned)groups);
    // waves a unit: as many as the card runs at once (and half as many again,
    // for experts that nobody chose), and runs of at most 8 quads.  Measured, gate/up +
    // down: 64 experts 3584 x 1792 at 64 rows with 4 + 2 waves 102 + 74 us,
    // with 2 + 2 123 + 74, with 4 + 4 102 + 87; 8 experts 3584 x 2560 at 64
    // rows, the layer with 4 waves 102 us, with 8 112; 64 experts 2048 x 1024 at
    // 4 rows with 4 waves 39 us, with 2 43, with 8 47.
    const size_t units = (size_t)grid.x * grid.y * grid.z;
    int waves = 1;
    while (waves < 8 && (2 * waves * units <= (size_t)1536 * OP::waves(RM) || plan.G > 8 * waves))
        waves *= 2;
    waves = std::min(waves, plan.S);
    const int L = plan.S / waves;
    size_t lds = (size_t)waves * tree_levels(L) * 4 * RM * 64 * sizeof(float);
    if (ch.parts)
        lds = std::max(lds, (size_t)(ch.M * ch.E + n) * sizeof(double));
    hipLaunchKernelGGL((q4_moe_product_kernel<OP, RM>), grid, dim3(64 * waves), lds, stream, ch, op, ids, weights,
                       wq, scales, L, plan);
    return hipGetLastError();
}

template <typename OP>
hipError_t launch_product(const Choice &ch, const OP &op, int *ids, float *weights, const uint8_t *wq,
                          const uint16_t *scales, const Plan &plan, hipStream_t stream)
{
    const int RM = row_group(ch.M * ch.topk, ch.E);
    if (RM == 1)
        return launch_product_r<OP, 1>(ch, op, ids, weights, wq, scales, plan, stream);
    if (RM == 2)
        return launch_product_r<OP, 2>(ch, op, ids, weights, wq, scales, plan, stream);
    return launch_product_r<OP, 4>(ch, op, ids, weights, wq, scales, plan, stream);
}

// The products of a piece of rows; ch.parts: the gate/up kernel chooses.
hipError_t products(const Choice &ch, const UpIn &x, int *ids, float *weights, const uint8_t *w13, const uint16_t *s13,
                    const uint8_t *w2, const uint16_t *s2, float *y, int I, const MoeRoom &room, hipStream_t stream)
{
    const int n = ch.M * ch.topk, H = x.H, shifts = MoeRoom::shifts_of(I);
    hipError_t e =
        x.lift ? launch_product(ch, Up<true>{x, room.hi, room.lo, room.shift, ch.topk, I, shifts}, ids, weights, w13,
                                s13, make_plan(H), stream)
               : launch_product(ch, Up<false>{x, room.hi, room.lo, room.shift, ch.topk, I, shifts}, ids, weights, w13,
                                s13, make_plan(H), stream);
    if (e != hipSuccess)
        return e;
    Choice given = ch;
    given.parts = nullptr;
    const Down down{{room.hi, room.lo, room.shift, n, I, shifts}, room.t, H};
    e = launch_product(given, down, ids, weights, w2, s2, make_plan(I), stream);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(q4_moe_join_kernel, dim3((unsigned)((H + 255) / 256), (unsigned)ch.M), dim3(64), 0, stream, ids,
                       weights, room.t, y, ch.topk, ch.E, H, ((uintptr_t)y & 15) == 0);
    return hipGetLastError();
}

}  // namespace

size_t moe_route_workspace_bytes(int M, int E, int K)
{
    return up256((size_t)logit_parts(M, E, K) * M * E * sizeof(double));
}

hipError_t launch_moe_route(const void *x, int x_kind, const void *router, int r_kind, const float *bias, int *ids,
                            float *weights, int M, int E, int K, int topk, int renormalize, void *workspace,
                            hipStream_t stream)
{
    double *parts = (double *)workspace;
    const hipError_t e = launch_logits(x, x_kind, router, r_kind, parts, Lifted{}, M, E, K, stream);
    if (e != hipSuccess)
        return e;
    const Choice ch{parts, bias, logit_parts(M, E, K), M, E, topk, renormalize};
    return launch_select(ch, ids, weights, nullptr, Lifted{}, K, stream);
}

size_t moe_workspace_bytes(int M, int H, int I, int topk)
{
    return MoeRoom(nullptr, chunk_rows(M, topk), topk, H, I).bytes;
}

hipError_t launch_moe_experts(const void *x, bool bf16, const int *ids, const float *weights, const uint8_t *w13,
                              const uint16_t *s13, const uint8_t *w2, const uint16_t *s2, float *y, int M, int topk,
                              int E, int H, int I, void *workspace, hipStream_t stream)
{
    const int rows = chunk_rows(M, topk);
    const MoeRoom room(workspace, rows, topk, H, I);
    for (int m = 0; m < M; m += rows) {
        const int now = std::min(rows, M - m);
        const uint16_t *xm = (const uint16_t *)x + (size_t)m * H;
        if (bf16) {
            hipLaunchKernelGGL(q4_moe_lift_kernel, dim3((unsigned)((now + 3) / 4)), dim3(256), 0, stream, xm, room.x,
                               now, H);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
        const Choice ch{nullptr, nullptr, 0, now, E, topk, 0};
        const hipError_t e = products(ch, room.in(xm, bf16, now, H), const_cast<int *>(ids) + (size_t)m * topk,
                                      const_cast<float *>(weights) + (size_t)m * topk, w13, s13, w2, s2,
                                      y + (size_t)m * H, I, room, stream);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// The whole layer's room: ids and weights, the logits' parts, the products'.
static size_t layer_room(int M, int E, int H, int topk)
{
    return 2 * up256((size_t)M * topk * 4) + moe_route_workspace_bytes(M, E, H);
}

size_t moe_layer_workspace_bytes(int M, int E, int H, int I, int topk)
{
    return layer_room(M, E, H, topk) + moe_workspace_bytes(M, H, I, topk);
}

hipError_t launch_moe_layer(const void *x, int x_kind, const void *router, int r_kind, const float *bias,
                            const uint8_t *w13, const uint16_t *s13, const uint8_t *w2, const uint16_t *s2, float *y,
                            int M, int E, int H, int I, int topk, int renormalize, void *workspace, hipStream_t stream)
{
    uint8_t *p = (uint8_t *)workspace;
    int *ids = (int *)p;
    float *weights = (float *)(p + up256((size_t)M * topk * 4));
    double *parts = (double *)(p + 2 * up256((size_t)M * topk * 4));
    void *rest = p + layer_room(M, E, H, topk);
    const bool bf16 = x_kind == 1;
    const int count = logit_parts(M, E, H);
    const Choice ch{parts, bias, count, M, E, topk, renormalize};
    if (chunk_rows(M, topk) < M) {  // too many rows for one piece
        const hipError_t e =
            launch_moe_route(x, x_kind, router, r_kind, bias, ids, weights, M, E, H, topk, renormalize, parts, stream);
        if (e != hipSuccess)
            return e;
        return launch_moe_experts(x, bf16, ids, weights, w13, s13, w2, s2, y, M, topk, E, H, I, rest, stream);
    }
    const MoeRoom room(rest, M, topk, H, I);
    const UpIn in = room.in(x, bf16, M, H);
    // x goes to binary16 beside the logits' parts, or beside the choice
    const bool by_rows = moe_by_rows(M, E, H);
    const bool fused = moe_fused(M, E, H);
    hipError_t e = launch_logits(x, x_kind, router, r_kind, parts, bf16 && !by_rows ? room.x : Lifted{}, M, E, H, stream);
    if (e != hipSuccess)
        return e;
    if (fused)
        return products(ch, in, ids, weights, w13, s13, w2, s2, y, I, room, stream);
    e = launch_select(ch, ids, weights, x, bf16 && by_rows ? room.x : Lifted{}, H, stream);
    if (e != hipSuccess)
        return e;
    const Choice given{nullptr, nullptr, 0, M, E, topk, 0};
    return products(given, in, ids, weights, w13, s13, w2, s2, y, I, room, stream);
}

}  // namespace q4
