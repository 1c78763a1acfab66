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
// each row and segment that puts its largest value in [2^14, 2^15): exact for
// every value down to 2^-31 of the largest, and off by at most 2^-40 of the
// largest below that, which a 32-bit sum cannot hold either.  h is kept as
// two binary16 numbers (the value and what its rounding left) after a power
// of two for each 32 values, 22 bits or more of each block's largest.  All
// sums are binary32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "q4_device.hpp"
#include "q4_launch.hpp"

namespace q4 {

namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kSlots = 1024;   // (row, choice) pairs one launch handles
constexpr int kExperts = 1024;  // most experts

// ---------------------------------------------------------------- router
// Sums in binary64 (v_mfma_f64_16x16x4): the choice compares neighbouring
// logits, and 32-bit sums would let their order decide it.
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

// grid = (16-expert tiles, 16-row tiles); the 16 waves take the chunks of 32 k
// in turn, and their sums are added in wave order.  Lane (g, c) holds expert
// c's (A) and row c's (B) values k = 32 s + 8 g + i of step i.
template <int XK, int RK>
__global__ __launch_bounds__(1024) void q4_moe_logits_kernel(const uint16_t *__restrict__ x,
                                                             const void *__restrict__ router,
                                                             const float *__restrict__ bias,
                                                             double *__restrict__ logits, int M, int E, int K)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int e = min((int)blockIdx.x * 16 + c, E - 1), m = min((int)blockIdx.y * 16 + c, M - 1);
    const uint16_t *xr = x + (size_t)m * K;
    const uint8_t *rr = (const uint8_t *)router + (size_t)e * K * (RK == 2 ? 4 : 2);
    f64x4 acc = {0, 0, 0, 0};
    for (int s = wave; s < K / 32; s += 16) {
        Eight<XK> a;
        Eight<RK> b;
        a.load(xr, 32 * (size_t)s + 8 * g);
        b.load(rr, 32 * (size_t)s + 8 * g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64(b.at(i), a.at(i), acc, 0, 0, 0);
    }
    __shared__ double part[16][4][64];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave >= 4)
        return;
    double s = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w)
        s += part[w][wave][lane];
    // component i of lane (g, c): expert 4 i + g of the tile, row c
    const int oe = blockIdx.x * 16 + 4 * wave + g, om = blockIdx.y * 16 + c;
    if (oe < E && om < M)
        logits[(size_t)om * E + oe] = s + (bias ? (double)bias[oe] : 0.0);
}

// One wave a row: every expert's rank is the number of experts before it (a
// larger logit, or the same at a lower index; NaN counts as the largest), and
// the first topk ranks are the choice.
__global__ __launch_bounds__(256) void q4_moe_select_kernel(const double *__restrict__ logits, int *__restrict__ ids,
                                                            float *__restrict__ weights, int E, int topk,
                                                            int renormalize)
{
    extern __shared__ double row[];  // E keys, then topk chosen logits
    double *chosen = row + E;
    const int m = blockIdx.x;
    const double *l = logits + (size_t)m * E;
    for (int e = threadIdx.x; e < E; e += 256)
        row[e] = l[e];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256) {
        const double v = row[e], key = v != v ? __builtin_inf() : v;
        int rank = 0;
        for (int f = 0; f < E; ++f) {
            const double u = row[f], k = u != u ? __builtin_inf() : u;
            rank += (k > key || (k == key && f < e)) ? 1 : 0;
        }
        if (rank < topk) {
            chosen[rank] = v;
            ids[(size_t)m * topk + rank] = v == -__builtin_inf() ? -1 : e;
        }
    }
    __syncthreads();
    if (threadIdx.x >= 64)
        return;
    const double top = chosen[0];
    // softmax over all experts, or over the chosen ones
    float sum = 0.f;
    const int n = renormalize ? topk : E;
    for (int i = threadIdx.x; i < n; i += 64) {
        const double v = renormalize ? chosen[i] : row[i];
        sum += v == -__builtin_inf() ? 0.f : __builtin_expf((float)(v - top));
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        sum += __shfl_xor(sum, d);
    for (int i = threadIdx.x; i < topk; i += 64) {
        const double v = chosen[i];
        weights[(size_t)m * topk + i] = v == -__builtin_inf() ? 0.f : __builtin_expf((float)(v - top)) / sum;
    }
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

__device__ __forceinline__ u32x4 load_codes(const uint8_t *p)
{
    return __builtin_nontemporal_load((const u32x4 *)p);
}
__device__ __forceinline__ u32x2 load_scales(const uint16_t *p)
{
    return __builtin_nontemporal_load((const u32x2 *)p);
}
__device__ __forceinline__ float quad_scale(u32x2 s, int j)
{
    return half_bits_to_float((j < 2 ? s.x : s.y) >> (16 * (j & 1)) & 0xFFFFu);
}

__device__ __forceinline__ f32x4 dot16(u32x4 a, u32x4 b, f32x4 c) { return blockdot_acc<false>(a, b, c); }

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

// The rows (slots) that chose expert e, in order, by one wave: -> count.
__device__ __forceinline__ int rows_of(const int *ids, int n, int e, uint16_t *list)
{
    const int lane = threadIdx.x & 63;
    int count = 0;
    for (int s0 = 0; s0 < n; s0 += 64) {
        const bool hit = s0 + lane < n && ids[s0 + lane] == e;
        const uint64_t mask = __ballot(hit);
        if (hit)
            list[count + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)(s0 + lane);
        count += __popcll(mask);
    }
    return count;
}

// gate and up.  grid = (I / 32, experts that can be chosen); wave j of a
// workgroup takes segment j of H for two tiles of gate and two of up, so the
// workgroup ends with 32 values of h, one block of the down product.
template <bool BF16, int R>
__global__ __launch_bounds__(1024) void q4_moe_up_kernel(const uint16_t *__restrict__ x, const int *__restrict__ ids,
                                                         const uint8_t *__restrict__ wq,
                                                         const uint16_t *__restrict__ scales, uint16_t *__restrict__ hi,
                                                         uint16_t *__restrict__ lo, int *__restrict__ shift, int n,
                                                         int topk, int E, int H, int I, Plan plan)
{
    extern __shared__ __attribute__((aligned(16))) float part[];  // [segment][tile][r][lane]
    __shared__ uint32_t seen[kExperts / 32];
    __shared__ uint16_t list[kSlots];
    __shared__ int found[2];  // the expert, its rows
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    if (wave == 0) {
        // the blockIdx.y-th of the chosen experts
        if (lane < kExperts / 32)
            seen[lane] = 0;
        __builtin_amdgcn_wave_barrier();
        for (int s = lane; s < n; s += 64) {
            const int e = ids[s];
            if (e >= 0 && e < E)
                atomicOr(&seen[e >> 5], 1u << (e & 31));
        }
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
        uint32_t bits = lane < kExperts / 32 ? ((volatile uint32_t *)seen)[lane] : 0;
        const int mine = __popc(bits);
        int before = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up(before, d);
            if (lane >= d)
                before += v;
        }
        before -= mine;
        int left = (int)blockIdx.y - before;
        if (lane == 0)
            found[0] = -1;
        __builtin_amdgcn_wave_barrier();
        if (lane < kExperts / 32 && left >= 0 && left < mine) {
            for (; left > 0; --left)
                bits &= bits - 1;
            found[0] = 32 * lane + __ffs(bits) - 1;
        }
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
        const int e = ((volatile int *)found)[0];
        const int count = e < 0 ? 0 : rows_of(ids, n, e, list);
        if (lane == 0)
            found[1] = count;
    }
    __syncthreads();
    const int e = found[0], count = found[1];
    if (e < 0)
        return;
    const int S = plan.S;
    const int qa = seg_first_block(plan, wave) / 4, qb = (seg_end_block(plan, wave) + 3) / 4;
    const Dequant<false> dq;
    // tiles: gate 2 t, gate 2 t + 1, up 2 t, up 2 t + 1 of the expert
    const size_t tile0 = (size_t)e * (2 * I / 16) + 2 * blockIdx.x;
    const uint8_t *w[4];
    const uint16_t *ws[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const size_t tile = tile0 + (t & 1) + (t >> 1) * (I / 16);
        w[t] = wq + tile * plan.G * 1024 + lane * 16;
        ws[t] = scales + tile * plan.G * 64 + c * 4;
    }
    for (int r0 = 0; r0 < count; r0 += 4 * R) {
        const int row = r0 + Slots<R>::row(c);
        const bool live = row < count;
        const uint16_t *xr = x + (size_t)(live ? list[row] / topk : 0) * H + 8 * g;
        auto load_x = [&](int o, int q) -> u32x4 {
            const int b = 4 * q + Slots<R>::block(o, c);
            if (live && b < plan.nb)
                return *(const u32x4 *)(xr + 32 * b);
            return (u32x4){0, 0, 0, 0};
        };
        int lift = 0;
        int back[R];
        if constexpr (BF16) {
            float top = 0.f;
            for (int q = qa; q < qb; ++q)
#pragma unroll
                for (int o = 0; o < R; ++o)
                    top = largest(load_x(o, q), top);
            // over the lanes that hold the same row: all four g, and the
            // slots of the row
            top = __builtin_fmaxf(top, __shfl_xor(top, 16));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            if constexpr (R == 1)
                top = __builtin_fmaxf(top, __shfl_xor(top, 1));
            if constexpr (R <= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, 2));
            lift = lift_of(top);
            // lane group g's rows are 4 r + g: slot 4 g + r holds row 4 r + g
#pragma unroll
            for (int r = 0; r < R; ++r)
                back[r] = __shfl(lift, 4 * g + r);
        }
        float p[4][R];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r)
                p[t][r] = 0.f;
        for (int q = qa; q < qb; ++q) {
            u32x4 a[R], codes[4];
            u32x2 sc[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                codes[t] = load_codes(w[t] + (size_t)q * 1024);
                sc[t] = load_scales(ws[t] + (size_t)q * 64);
            }
#pragma unroll
            for (int o = 0; o < R; ++o) {
                a[o] = load_x(o, q);
                if constexpr (BF16)
                    a[o] = lifted(a[o], lift);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 D[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    D[j] = blockdot<false>(a[Slots<R>::operand(j)], dq(codes[t][j]));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = quad_scale(sc[t], j);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        p[t][r] = __builtin_fmaf(d, D[j][Slots<R>::comp(j, r)], p[t][r]);
                }
            }
        }
        if (r0)
            __syncthreads();  // the last group's sums are read
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float v = p[t][r];
                if constexpr (BF16)
                    v = __builtin_ldexpf(v, -back[r]);
                part[((wave * 4 + t) * R + r) * 64 + lane] = v;
            }
        __syncthreads();
        // 32 lanes a row: the trees, the activation, the block's power of two
        const int rows = min(count - r0, 4 * R);
        for (int o = threadIdx.x; o < rows * 32; o += blockDim.x) {
            const int i = o >> 5, col = o & 31;
            const int at = ((col >> 4) * R + (i >> 2)) * 64 + (i & 3) * 16 + (col & 15);
            float gv[16], uv[16];
#pragma unroll
            for (int s = 0; s < 16; ++s) {
                gv[s] = s < S ? part[s * 4 * R * 64 + at] : 0.f;
                uv[s] = s < S ? part[s * 4 * R * 64 + 2 * R * 64 + at] : 0.f;
            }
            const float gate = tree_sum<16>(gv, S), up = tree_sum<16>(uv, S);
            const float h = gate / (1.f + __builtin_expf(-gate)) * up;
            float top = __builtin_fabsf(h) < __builtin_inff() ? __builtin_fabsf(h) : 0.f;
#pragma unroll
            for (int d = 1; d < 32; d *= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, d));
            const int up2 = lift_of(top);
            const float v = __builtin_ldexpf(h, up2);
            const _Float16 vh = (_Float16)v;
            const float rest = v - (float)vh;
            const _Float16 vl = __builtin_fabsf(v) < __builtin_inff() ? (_Float16)rest : (_Float16)0.f;
            const size_t slot = list[r0 + i];
            const size_t k = slot * I + 32 * blockIdx.x + col;
            hi[k] = __builtin_bit_cast(uint16_t, vh);
            lo[k] = __builtin_bit_cast(uint16_t, vl);
            if (col == 0)
                shift[slot * (I / 32) + blockIdx.x] = -up2;
        }
    }
}

// down and the sum over the chosen experts.  grid = tiles of 16 columns of y;
// a workgroup's waves take (expert, run of segments) pairs in turn, the runs'
// roots meet in LDS, and each output adds its experts in the order of j.
template <int R>
__global__ __launch_bounds__(1024) void q4_moe_down_kernel(const int *__restrict__ ids,
                                                           const float *__restrict__ weights,
                                                           const uint16_t *__restrict__ hi,
                                                           const uint16_t *__restrict__ lo,
                                                           const int *__restrict__ shift,
                                                           const uint8_t *__restrict__ wq,
                                                           const uint16_t *__restrict__ scales, float *__restrict__ y,
                                                           int M, int topk, int E, int H, int I, Plan plan)
{
    extern __shared__ __attribute__((aligned(16))) float root[];  // [slot][run][16 columns]
    __shared__ int first[kExperts];      // an expert's rows before the scatter, their end after it
    __shared__ uint16_t list[kSlots];    // slots in the order of their experts
    __shared__ uint16_t active[kExperts];  // chosen experts
    __shared__ int sums[2][16];
    __shared__ int total;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int n = M * topk;
    // counting sort of the slots by expert
    first[tid] = 0;
    __syncthreads();
    const int id = tid < n ? ids[tid] : -1;
    const bool valid = id >= 0 && id < E;
    if (valid)
        atomicAdd(&first[id], 1);
    __syncthreads();
    const int count = first[tid];
    int before = count, rank = count > 0;
    for (int d = 1; d < 64; d *= 2) {
        const int a = __shfl_up(before, d), b = __shfl_up(rank, d);
        if (lane >= d) {
            before += a;
            rank += b;
        }
    }
    if (lane == 63) {
        sums[0][wave] = before;
        sums[1][wave] = rank;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        before += sums[0][w];
        rank += sums[1][w];
    }
    if (count)
        active[rank - 1] = (uint16_t)tid;
    first[tid] = before - count;
    if (tid == 1023)
        total = rank;
    __syncthreads();
    // (the order of an expert's rows in the list does not matter: a row's bits
    // do not depend on its place)
    if (valid)
        list[atomicAdd(&first[id], 1)] = (uint16_t)tid;
    __syncthreads();
    const int A = total, S = plan.S;
    int runs = 1;
    while (A * runs < 16 && 2 * runs <= S && 2 * runs * n <= kSlots)
        runs *= 2;
    const int L = S / runs;
    const Dequant<false> dq;
    for (int u = wave; u < A * runs; u += 16) {
        const int e = active[u / runs], run = u % runs;
        const int end = first[e], begin = u / runs ? first[active[u / runs - 1]] : 0;
        const size_t tile = (size_t)e * (H / 16) + blockIdx.x;
        const uint8_t *w = wq + tile * plan.G * 1024 + lane * 16;
        const uint16_t *ws = scales + tile * plan.G * 64 + c * 4;
        for (int r0 = begin; r0 < end; r0 += 4 * R) {
            const int row = r0 + Slots<R>::row(c);
            const bool live = row < end;
            const size_t slot = live ? list[row] : 0;
            const uint16_t *ph = hi + slot * I + 8 * g, *pl = lo + slot * I + 8 * g;
            // the rows whose values this lane group accumulates
            const int *sh[R];
            int mine[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int i = r0 + 4 * r + g;
                mine[r] = i < end ? list[i] : -1;
                sh[r] = shift + (size_t)max(mine[r], 0) * (I / 32);
            }
            TreeStack<R, float> tree;
            float p[R];
            for (int li = 0; li < L; ++li) {
                const int s = run * L + li;
                const int qa = seg_first_block(plan, s) / 4, qb = (seg_end_block(plan, s) + 3) / 4;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    p[r] = 0.f;
                for (int q = qa; q < qb; ++q) {
                    const u32x4 codes = load_codes(w + (size_t)q * 1024);
                    const u32x2 sc = load_scales(ws + (size_t)q * 64);
                    u32x4 ah[R], al[R];
#pragma unroll
                    for (int o = 0; o < R; ++o) {
                        const int b = 4 * q + Slots<R>::block(o, c);
                        ah[o] = al[o] = (u32x4){0, 0, 0, 0};
                        if (live && b < plan.nb) {
                            ah[o] = *(const u32x4 *)(ph + 32 * b);
                            al[o] = *(const u32x4 *)(pl + 32 * b);
                        }
                    }
                    f32x4 D[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x4 b = dq(codes[j]);
                        D[j] = dot16(ah[Slots<R>::operand(j)], b, blockdot<false>(al[Slots<R>::operand(j)], b));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (4 * q + j < plan.nb) {
                            const float d = quad_scale(sc, j);
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                p[r] = __builtin_fmaf(__builtin_ldexpf(d, sh[r][4 * q + j]),
                                                      D[j][Slots<R>::comp(j, r)], p[r]);
                        }
                    }
                }
                tree.push(p, li, L);
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (mine[r] >= 0)
                    root[(mine[r] * runs + run) * 16 + c] = p[r];
        }
    }
    __syncthreads();
    for (int o = tid; o < M * 16; o += 1024) {
        const int m = o >> 4, col = o & 15;
        float sum = 0.f;
        for (int j = 0; j < topk; ++j) {
            const int slot = m * topk + j, x = ids[slot];
            if (x < 0 || x >= E)
                continue;
            float v[16];
#pragma unroll
            for (int s = 0; s < 16; ++s)
                v[s] = s < runs ? root[(slot * runs + s) * 16 + col] : 0.f;
            sum = __builtin_fmaf(weights[slot], tree_sum<16>(v, runs), sum);
        }
        y[(size_t)m * H + 16 * blockIdx.x + col] = sum;
    }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Rows one launch handles.
int chunk_rows(int M, int topk) { return std::min(M, kSlots / topk); }

template <int XK>
void launch_logits(int rk, dim3 grid, const uint16_t *x, const void *router, const float *bias, double *logits, int M,
                   int E, int K, hipStream_t stream)
{
    if (rk == 2)
        hipLaunchKernelGGL((q4_moe_logits_kernel<XK, 2>), grid, dim3(1024), 0, stream, x, router, bias, logits, M, E, K);
    else
        hipLaunchKernelGGL((q4_moe_logits_kernel<XK, XK>), grid, dim3(1024), 0, stream, x, router, bias, logits, M, E,
                           K);
}

template <bool BF16, int R>
hipError_t launch_experts(const uint16_t *x, const int *ids, const float *weights, const uint8_t *w13,
                          const uint16_t *s13, const uint8_t *w2, const uint16_t *s2, float *y, int M, int topk, int E,
                          int H, int I, uint16_t *hi, uint16_t *lo, int *shift, hipStream_t stream)
{
    const Plan up = make_plan(H), down = make_plan(I);
    const int n = M * topk;
    const size_t lds_up = (size_t)up.S * 4 * R * 64 * sizeof(float);
    // (the largest with the kernels' fixed parts passes the default limit)
    hipError_t e = hipSuccess;
    if (R == 4)
        e = hipFuncSetAttribute((const void *)q4_moe_up_kernel<BF16, R>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)lds_up);
    // roots: [slot][run][16], where the kernel keeps slots x runs within kSlots
    const size_t lds_down = (size_t)std::min(kSlots, 16 * n) * 16 * sizeof(float);
    if (e == hipSuccess && lds_down > 32 * 1024)
        e = hipFuncSetAttribute((const void *)q4_moe_down_kernel<R>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)lds_down);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((q4_moe_up_kernel<BF16, R>), dim3((unsigned)(I / 32), (unsigned)std::min(n, E)),
                       dim3(64 * up.S), lds_up, stream, x, ids, w13, s13, hi, lo, shift, n, topk, E, H, I, up);
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((q4_moe_down_kernel<R>), dim3((unsigned)(H / 16)), dim3(1024), lds_down, stream, ids, weights,
                       hi, lo, shift, w2, s2, y, M, topk, E, H, I, down);
    return hipGetLastError();
}

}  // namespace

size_t moe_route_workspace_bytes(int M, int E) { return up256((size_t)M * E * sizeof(double)); }

hipError_t launch_moe_route(const void *x, int x_kind, const void *router, int r_kind, const float *bias, int *ids,
                            float *weights, int M, int E, int K, int topk, int renormalize, void *workspace,
                            hipStream_t stream)
{
    double *logits = (double *)workspace;
    const dim3 grid((unsigned)((E + 15) / 16), (unsigned)((M + 15) / 16));
    if (x_kind == 1)
        launch_logits<1>(r_kind, grid, (const uint16_t *)x, router, bias, logits, M, E, K, stream);
    else
        launch_logits<0>(r_kind, grid, (const uint16_t *)x, router, bias, logits, M, E, K, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(q4_moe_select_kernel, dim3((unsigned)M), dim3(256), (size_t)(E + topk) * sizeof(double), stream,
                       logits, ids, weights, E, topk, renormalize);
    return hipGetLastError();
}

size_t moe_workspace_bytes(int M, int I, int topk)
{
    const size_t n = (size_t)chunk_rows(M, topk) * topk;
    return 2 * up256(n * I * sizeof(uint16_t)) + up256(n * (I / 32) * sizeof(int));
}

hipError_t launch_moe_experts(const void *x, bool bf16, const int *ids, const float *weights, const uint8_t *w13,
                              const uint16_t *s13, const uint8_t *w2, const uint16_t *s2, float *y, int M, int topk,
                              int E, int H, int I, void *workspace, hipStream_t stream)
{
    const int rows = chunk_rows(M, topk);
    const size_t part = up256((size_t)rows * topk * I * sizeof(uint16_t));
    uint16_t *hi = (uint16_t *)workspace;
    uint16_t *lo = (uint16_t *)((uint8_t *)workspace + part);
    int *shift = (int *)((uint8_t *)workspace + 2 * part);
    for (int m = 0; m < M; m += rows) {
        const int now = std::min(rows, M - m);
        const uint16_t *xm = (const uint16_t *)x + (size_t)m * H;
        const int *im = ids + (size_t)m * topk;
        const float *wm = weights + (size_t)m * topk;
        float *ym = y + (size_t)m * H;
        hipError_t e;
#define Q4_MOE(B, R) launch_experts<B, R>(xm, im, wm, w13, s13, w2, s2, ym, now, topk, E, H, I, hi, lo, shift, stream)
        if (now <= 4)
            e = bf16 ? Q4_MOE(true, 1) : Q4_MOE(false, 1);
        else if (now <= 8)
            e = bf16 ? Q4_MOE(true, 2) : Q4_MOE(false, 2);
        else
            e = bf16 ? Q4_MOE(true, 4) : Q4_MOE(false, 4);
#undef Q4_MOE
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace q4
