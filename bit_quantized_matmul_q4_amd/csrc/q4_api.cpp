// q4_api.cpp -- the C ABI of libq4.so (declared in include/q4.h).
//
// Argument checks, the crossover dispatcher and status codes.  The kernel
// choice follows the row-count switch of "Why Continuous Batching Slowed
// Down My LLM Inference Engine: A Metal Kernel Investigation" (section "Two
// Rows of Input, Two Different Kernels": one row -> matrix-vector, more ->
// matrix-matrix; section "Row-by-Row GEMV to the Rescue": the switch moved to
// a measured threshold, <= 4 rows -> matrix-vector).  Here the threshold is
// the crossover measured on MI355X, and because both kernels share one
// reduction order the choice changes speed only, never the bits.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include <hip/hip_runtime_api.h>

#include "../../include/q4.h"
#include "q4_launch.hpp"
#include "q4_plan.hpp"

namespace {

// Measured GEMV -> GEMM crossover on MI355X (rows); M <= T runs the GEMV.
// On the Qwen2.5-7B-shaped layer set (the sum of the six projections' times)
// the matrix-matrix kernel first wins at M = 17, where the matrix-vector
// kernel needs a second 16-row slice (102 vs 106 us); at 16 the matrix-vector
// kernel is 10% faster (73 vs 81 us).  T = 16.
constexpr int kDefaultCrossover = 16;
// Long K (K > 8192), measured: the matrix-vector kernel's time grows with the
// rows (down_proj 3584 x 18944: 16.9 us at 9 rows, 23.2 at 16) while the
// matrix-matrix kernel, split over K, stays near 16 us; from 9 rows on it is
// faster, provided it gets its split workspace (without it, down_proj takes
// several times longer).
constexpr int kLongK = 8192, kLongKCrossover = 8;

thread_local int g_last_hip = 0;

int env_int(const char *name, int fallback)
{
    const char *v = std::getenv(name);
    if (!v || !*v)
        return fallback;
    char *end = nullptr;
    const long r = std::strtol(v, &end, 10);
    if (end == v || *end != '\0' || r < 0 || r > (1 << 30))
        return fallback;
    return (int)r;
}

std::atomic<int> &crossover()
{
    static std::atomic<int> t{env_int("Q4_CROSSOVER", kDefaultCrossover)};
    return t;
}

// Q4_KERNEL=gemv|gemm forces a kernel for Q4_AUTO calls (read once).
int forced_kernel()
{
    static const int k = [] {
        const char *v = std::getenv("Q4_KERNEL");
        if (v && std::strcmp(v, "gemv") == 0)
            return (int)Q4_GEMV;
        if (v && std::strcmp(v, "gemm") == 0)
            return (int)Q4_GEMM;
        return (int)Q4_AUTO;
    }();
    return k;
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_shape(long long M, long long N, long long K)
{
    if (M < 1 || N < 1 || K < 32 || K % 32 != 0)
        return Q4_ERR_SHAPE;
    // one column tile's packed codes (K / 2 * 16 bytes) and 16 rows of x
    // (32 K bytes) stay below 2^31 bytes: the kernels address them with
    // 32-bit offsets
    if (K > (1LL << 25))
        return Q4_ERR_SHAPE;
    // every element count must fit comfortably in 63 bits and every row
    // index product used by the kernels in size_t
    const long long lim = 1LL << 46;
    if (M > lim / K || N > lim / K || M > lim / N)
        return Q4_ERR_SHAPE;
    return Q4_OK;
}

// Shapes of the 8-bit product: the 32-bit sums stay exact (K 2^14 < 2^31, for
// codes down to -128), and every launch stays below 2^32 threads.
int check_int8(long long rows, long long N, long long K)
{
    if (rows < 1 || N < 1 || K < 32 || K % 32 != 0 || K > Q4_INT8_MAX_K)
        return Q4_ERR_SHAPE;
    const long long lim = 1LL << 24;
    if (rows > lim || N > lim || rows > (1LL << 36) / N)
        return Q4_ERR_SHAPE;
    return Q4_OK;
}

// Shapes of the expert layer: what its grids and 32-bit offsets hold.
int check_moe(long long M, long long E, long long K, long long topk)
{
    if (M < 1 || E < 1 || topk < 1 || topk > E || K < 32 || K % 32 != 0)
        return Q4_ERR_SHAPE;
    if (M > Q4_MOE_MAX_ROWS || E > Q4_MOE_MAX_EXPERTS || K > (1LL << 17))
        return Q4_ERR_SHAPE;
    return Q4_OK;
}

// Shapes of the microscaled 4-bit form and its product.
int check_mx4(long long rows, long long N, long long K)
{
    if (rows < 1 || N < 1 || K < 32 || K % 32 != 0 || K > Q4_MX4_MAX_K)
        return Q4_ERR_SHAPE;
    const long long lim = 1LL << 24;
    if (rows > lim || N > lim || rows > (1LL << 36) / N)
        return Q4_ERR_SHAPE;
    return Q4_OK;
}

bool is_float(int dtype) { return dtype == Q4_F16 || dtype == Q4_BF16 || dtype == Q4_F32; }

// The launchers' element kinds.
int elem_kind(int dtype) { return dtype == Q4_F32 ? 2 : dtype == Q4_BF16 ? 1 : 0; }

int hip_status(hipError_t e)
{
    if (e == hipSuccess)
        return Q4_OK;
    g_last_hip = (int)e;
    return Q4_ERR_HIP;
}

}  // namespace

extern "C" {

int q4_abi_version(void) { return Q4_ABI_VERSION; }

int q4_last_hip_error(void) { return g_last_hip; }

const char *q4_strerror(int status)
{
    switch (status) {
    case Q4_OK: return "ok";
    case Q4_ERR_NULL: return "a required pointer is NULL";
    case Q4_ERR_SHAPE: return "bad shape (need M >= 1, N >= 1, K >= 32, K % 32 == 0, 1 <= topk <= experts, eps >= 0, sizes in range)";
    case Q4_ERR_ALIGN: return "misaligned pointer (x, Wq, router, quantizer w and codes: 16 B; packed scales: 8 B, microscaled 4 B; y, float32 scales, bias, ids, weights: 4 B; 16-bit y: 2 B; q4_block_norm: its elements'; workspace: 256 B)";
    case Q4_ERR_ENUM: return "unknown dtype, kernel selector, norm kind or gate form";
    case Q4_ERR_HIP: return "HIP launch error (see q4_last_hip_error)";
    case Q4_ERR_WORKSPACE: return "workspace too small or absent in a call that needs one, or workspace_bytes > 0 with a NULL workspace";
    case Q4_ERR_SCRATCH: return "the call needs more than the library's fixed scratch buffer (Q4_SCRATCH_BYTES)";
    default: return "unknown status";
    }
}

int q4_get_crossover(void) { return crossover().load(std::memory_order_relaxed); }

int q4_set_crossover(int T)
{
    if (T < 0)
        return Q4_ERR_SHAPE;
    crossover().store(T, std::memory_order_relaxed);
    return Q4_OK;
}

int q4_segments(int K)
{
    if (K < 32 || K % 32 != 0)
        return 0;
    return q4::make_plan(K).S;
}

// The kernel Q4_AUTO runs: matrix-vector iff M <= T, except that for
// K > kLongK the matrix-matrix kernel already runs above min(T, 8) rows when
// it has the workspace it asks for (ws_ok).
static int auto_kernel(int M, int K, bool ws_ok)
{
    if (forced_kernel() != Q4_AUTO)
        return forced_kernel();
    const int T = q4_get_crossover();
    if (M > T)
        return Q4_GEMM;
    if (K > kLongK && M > std::min(T, kLongKCrossover) && ws_ok)
        return Q4_GEMM;
    return Q4_GEMV;
}

size_t q4_workspace_bytes(int M, int N, int K, int kernel)
{
    if (check_shape(M, N, K) != Q4_OK)
        return 0;
    const int k = kernel == Q4_AUTO ? auto_kernel(M, K, true) : kernel;
    if (k != Q4_GEMM)
        return 0;
    return q4::gemm_workspace_bytes(M, N, K);
}

// The checks and dispatch shared by q4_linear_ex and q4_linear_noalloc.
// scratch: take the library's fixed device buffer as the workspace (the
// caller passes none).
static int linear_impl(const void *x, int x_dtype, const void *Wq, const void *scales, float *y, int M, int N,
                       int K, int kernel, void *workspace, size_t workspace_bytes, bool scratch, void *stream)
{
    if (!x || !Wq || !scales || !y)
        return Q4_ERR_NULL;
    if (x_dtype != Q4_F16 && x_dtype != Q4_BF16)
        return Q4_ERR_ENUM;
    if (kernel != Q4_AUTO && kernel != Q4_GEMV && kernel != Q4_GEMM)
        return Q4_ERR_ENUM;
    const int sh = check_shape(M, N, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(x, 16) || !aligned(Wq, 16) || !aligned(scales, 8) || !aligned(y, 4))
        return Q4_ERR_ALIGN;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;

    const size_t need = q4::gemm_workspace_bytes(M, N, K);
    const int k = kernel == Q4_AUTO
                      ? auto_kernel(M, K, scratch ? need <= q4::kScratchBytes : workspace_bytes >= need)
                      : kernel;
    if (k == Q4_GEMM && scratch) {
        if (need > q4::kScratchBytes)
            return Q4_ERR_SCRATCH;
        if (need > 0) {
            const int st = hip_status(q4::scratch_buffer(&workspace));
            if (st != Q4_OK)
                return st;
            workspace_bytes = need;
        }
    }

    const bool bf16 = x_dtype == Q4_BF16;
    hipStream_t s = (hipStream_t)stream;
    if (k == Q4_GEMV)
        return hip_status(q4::launch_gemv(x, bf16, (const uint8_t *)Wq, (const uint16_t *)scales, y,
                                          M, N, K, s));
    return hip_status(q4::launch_gemm(x, bf16, (const uint8_t *)Wq, (const uint16_t *)scales, y, M, N,
                                      K, workspace_bytes ? workspace : nullptr, workspace_bytes, s));
}

int q4_linear_ex(const void *x, int x_dtype, const void *Wq, const void *scales, float *y,
                 int M, int N, int K, int kernel, void *workspace, size_t workspace_bytes,
                 void *stream)
{
    return linear_impl(x, x_dtype, Wq, scales, y, M, N, K, kernel, workspace, workspace_bytes, false, stream);
}

int q4_linear_noalloc(const void *x, int x_dtype, const void *Wq, const void *scales, float *y, int M, int N,
                      int K, int kernel, void *stream)
{
    return linear_impl(x, x_dtype, Wq, scales, y, M, N, K, kernel, nullptr, 0, true, stream);
}

int q4_linear(const void *x, const void *Wq, const void *scales, float *y, int M, int N, int K,
              void *stream)
{
    return q4_linear_ex(x, Q4_BF16, Wq, scales, y, M, N, K, Q4_AUTO, nullptr, 0, stream);
}

int q4_linear_f16(const void *x, const void *Wq, const void *scales, float *y, int M, int N, int K,
                  void *stream)
{
    return q4_linear_ex(x, Q4_F16, Wq, scales, y, M, N, K, Q4_AUTO, nullptr, 0, stream);
}

size_t q4_packed_code_bytes(int N, int K)
{
    if (check_shape(1, N, K) != Q4_OK)
        return 0;
    return q4::packed_code_bytes(N, K);
}

size_t q4_packed_scale_bytes(int N, int K)
{
    if (check_shape(1, N, K) != Q4_OK)
        return 0;
    return q4::packed_scale_bytes(N, K);
}

int q4_quantize(const void *w, int w_dtype, uint8_t *codes, void *scales, int N, int K, void *stream)
{
    if (!w || !codes || !scales)
        return Q4_ERR_NULL;
    if (w_dtype != Q4_F16 && w_dtype != Q4_BF16 && w_dtype != Q4_F32)
        return Q4_ERR_ENUM;
    const int sh = check_shape(1, N, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 2))
        return Q4_ERR_ALIGN;
    const int kind = w_dtype == Q4_F32 ? 2 : w_dtype == Q4_BF16 ? 1 : 0;
    return hip_status(q4::launch_quantize(w, kind, codes, (uint16_t *)scales, N, K, (hipStream_t)stream));
}

static int pack_impl(const uint8_t *codes, bool nibbles, const void *scales, uint8_t *Wq, void *Wscales, int N,
                     int K, void *stream)
{
    if (!codes || !scales || !Wq || !Wscales)
        return Q4_ERR_NULL;
    const int sh = check_shape(1, N, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(scales, 2) || !aligned(Wq, 16) || !aligned(Wscales, 8))
        return Q4_ERR_ALIGN;
    return hip_status(q4::launch_pack(codes, nibbles, (const uint16_t *)scales, Wq, (uint16_t *)Wscales, N, K,
                                      (hipStream_t)stream));
}

int q4_pack(const uint8_t *codes, const void *scales, uint8_t *Wq, void *Wscales, int N, int K,
            void *stream)
{
    return pack_impl(codes, false, scales, Wq, Wscales, N, K, stream);
}

int q4_pack_nibbles(const uint8_t *Wq_rows, const void *scales, uint8_t *Wq, void *Wscales, int N, int K,
                    void *stream)
{
    return pack_impl(Wq_rows, true, scales, Wq, Wscales, N, K, stream);
}

int q4_linear_grouped(const void *x, int x_dtype, const q4_group_item *items, int count, int M, int K,
                      void *workspace, size_t workspace_bytes, void *stream)
{
    if (!x || !items)
        return Q4_ERR_NULL;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;
    if (x_dtype != Q4_F16 && x_dtype != Q4_BF16)
        return Q4_ERR_ENUM;
    if (count < 1 || count > Q4_GROUP_MAX)
        return Q4_ERR_SHAPE;
    if (!aligned(x, 16))
        return Q4_ERR_ALIGN;
    q4::GroupItem g[Q4_GROUP_MAX];
    for (int i = 0; i < count; ++i) {
        const q4_group_item &it = items[i];
        if (!it.Wq || !it.scales || !it.y)
            return Q4_ERR_NULL;
        const int sh = check_shape(M, it.N, K);
        if (sh != Q4_OK)
            return sh;
        if (!aligned(it.Wq, 16) || !aligned(it.scales, 8) || !aligned(it.y, 4))
            return Q4_ERR_ALIGN;
        g[i] = q4::GroupItem{(const uint8_t *)it.Wq, (const uint16_t *)it.scales, it.y, it.N};
    }
    const bool bf16 = x_dtype == Q4_BF16;
    hipStream_t s = (hipStream_t)stream;
    // one launch of the matrix-vector kernel where the crossover rule picks
    // it for every matrix (as q4_linear_ex with Q4_AUTO and this workspace
    // would); otherwise, and for groups too wide for one launch, each matrix
    // as q4_linear_ex (the calls are stream-ordered, so they can share the
    // workspace)
    bool ws_ok = workspace != nullptr;
    for (int i = 0; i < count; ++i)
        ws_ok = ws_ok && q4::gemm_workspace_bytes(M, g[i].N, K) <= workspace_bytes;
    if (auto_kernel(M, K, ws_ok) == Q4_GEMV) {
        hipError_t e = hipSuccess;
        if (q4::launch_gemv_grouped(x, bf16, g, count, M, K, s, &e))
            return hip_status(e);
    }
    for (int i = 0; i < count; ++i) {
        const int st = linear_impl(x, x_dtype, g[i].wq, g[i].scales, g[i].y, M, g[i].N, K, Q4_AUTO, workspace,
                                   workspace_bytes, false, stream);
        if (st != Q4_OK)
            return st;
    }
    return Q4_OK;
}

size_t q4_int8_packed_bytes(int rows, int K)
{
    return check_int8(rows, 1, K) == Q4_OK ? q4::int8_packed_bytes(rows, K) : 0;
}

static int int8_quantize_impl(const void *w, int w_dtype, int8_t *codes, bool packed, float *scales, int rows, int K,
                              void *stream)
{
    if (!w || !codes || !scales)
        return Q4_ERR_NULL;
    if (w_dtype != Q4_F16 && w_dtype != Q4_BF16 && w_dtype != Q4_F32)
        return Q4_ERR_ENUM;
    const int sh = check_int8(rows, 1, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return Q4_ERR_ALIGN;
    return hip_status(
        q4::launch_int8_quantize(w, elem_kind(w_dtype), codes, packed, scales, rows, K, (hipStream_t)stream));
}

int q4_int8_quantize(const void *w, int w_dtype, int8_t *codes, float *scales, int rows, int K, void *stream)
{
    return int8_quantize_impl(w, w_dtype, codes, false, scales, rows, K, stream);
}

int q4_int8_quantize_pack(const void *w, int w_dtype, void *packed, float *scales, int rows, int K, void *stream)
{
    return int8_quantize_impl(w, w_dtype, (int8_t *)packed, true, scales, rows, K, stream);
}

int q4_int8_pack(const int8_t *codes, void *packed, int rows, int K, void *stream)
{
    if (!codes || !packed)
        return Q4_ERR_NULL;
    const int sh = check_int8(rows, 1, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(codes, 16) || !aligned(packed, 16))
        return Q4_ERR_ALIGN;
    return hip_status(q4::launch_int8_pack(codes, (int8_t *)packed, rows, K, (hipStream_t)stream));
}

size_t q4_int8_workspace_bytes(int M, int N, int K, int x_dtype)
{
    if (check_int8(M, N, K) != Q4_OK || (x_dtype != Q4_F16 && x_dtype != Q4_BF16 && x_dtype != Q4_I8))
        return 0;
    return q4::int8_workspace_bytes(x_dtype != Q4_I8, M, N, K);
}

int q4_int8_linear(const void *x, int x_dtype, const float *x_scales, const void *Wq, const float *w_scales, void *y,
                   int y_dtype, int M, int N, int K, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!x || !Wq || !w_scales || !y || (x_dtype == Q4_I8 && !x_scales))
        return Q4_ERR_NULL;
    if (x_dtype != Q4_F16 && x_dtype != Q4_BF16 && x_dtype != Q4_I8)
        return Q4_ERR_ENUM;
    if (y_dtype != Q4_F16 && y_dtype != Q4_BF16 && y_dtype != Q4_F32)
        return Q4_ERR_ENUM;
    const int sh = check_int8(M, N, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(x, 16) || !aligned(Wq, 16) || !aligned(w_scales, 4) || !aligned(y, y_dtype == Q4_F32 ? 4 : 2) ||
        (x_dtype == Q4_I8 && !aligned(x_scales, 4)))
        return Q4_ERR_ALIGN;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::int8_workspace_bytes(x_dtype != Q4_I8, M, N, K))
        return Q4_ERR_WORKSPACE;
    return hip_status(q4::launch_int8_linear(x, x_dtype == Q4_I8 ? -1 : elem_kind(x_dtype), x_scales,
                                             (const int8_t *)Wq, w_scales, y, elem_kind(y_dtype), M, N, K, workspace,
                                             (hipStream_t)stream));
}

size_t q4_mx4_code_bytes(int rows, int K)
{
    return check_mx4(rows, 1, K) == Q4_OK ? q4::mx4_code_bytes(rows, K) : 0;
}

size_t q4_mx4_scale_bytes(int rows, int K)
{
    return check_mx4(rows, 1, K) == Q4_OK ? q4::mx4_scale_bytes(rows, K) : 0;
}

static int mx4_quantize(const void *w, int w_dtype, uint8_t *codes, uint8_t *scales, bool packed, int rows, int K,
                        void *stream)
{
    if (!w || !codes || !scales)
        return Q4_ERR_NULL;
    if (!is_float(w_dtype))
        return Q4_ERR_ENUM;
    const int sh = check_mx4(rows, 1, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(w, 16) || !aligned(codes, 16) || (packed && !aligned(scales, 4)))
        return Q4_ERR_ALIGN;
    return hip_status(q4::launch_mx4_quantize(w, elem_kind(w_dtype), codes, scales, packed, rows, K,
                                              (hipStream_t)stream));
}

int q4_mx4_quantize(const void *w, int w_dtype, uint8_t *codes, uint8_t *scales, int rows, int K, void *stream)
{
    return mx4_quantize(w, w_dtype, codes, scales, false, rows, K, stream);
}

int q4_mx4_quantize_pack(const void *w, int w_dtype, void *packed, void *packed_scales, int rows, int K, void *stream)
{
    return mx4_quantize(w, w_dtype, (uint8_t *)packed, (uint8_t *)packed_scales, true, rows, K, stream);
}

int q4_mx4_pack(const uint8_t *codes, const uint8_t *scales, void *packed, void *packed_scales, int rows, int K,
                void *stream)
{
    if (!codes || !scales || !packed || !packed_scales)
        return Q4_ERR_NULL;
    const int sh = check_mx4(rows, 1, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(codes, 16) || !aligned(packed, 16) || !aligned(packed_scales, 4))
        return Q4_ERR_ALIGN;
    return hip_status(q4::launch_mx4_pack(codes, scales, (uint8_t *)packed, (uint8_t *)packed_scales, rows, K,
                                          (hipStream_t)stream));
}

int q4_mx4_dequantize(const void *packed, const void *packed_scales, void *w, int w_dtype, int rows, int K,
                      void *stream)
{
    if (!packed || !packed_scales || !w)
        return Q4_ERR_NULL;
    if (!is_float(w_dtype))
        return Q4_ERR_ENUM;
    const int sh = check_mx4(rows, 1, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(packed, 16) || !aligned(packed_scales, 4) || !aligned(w, 16))
        return Q4_ERR_ALIGN;
    return hip_status(q4::launch_mx4_dequantize((const uint8_t *)packed, (const uint8_t *)packed_scales, w,
                                                elem_kind(w_dtype), rows, K, (hipStream_t)stream));
}

size_t q4_mx4_workspace_bytes(int M, int N, int K, int x_dtype)
{
    if (check_mx4(M, N, K) != Q4_OK || (x_dtype != Q4_F16 && x_dtype != Q4_BF16 && x_dtype != Q4_MX4))
        return 0;
    return q4::mx4_workspace_bytes(x_dtype != Q4_MX4, M, N, K);
}

int q4_mx4_linear(const void *x, int x_dtype, const void *x_scales, const void *Wq, const void *w_scales, void *y,
                  int y_dtype, int M, int N, int K, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!x || !Wq || !w_scales || !y || (x_dtype == Q4_MX4 && !x_scales))
        return Q4_ERR_NULL;
    if ((x_dtype != Q4_F16 && x_dtype != Q4_BF16 && x_dtype != Q4_MX4) || !is_float(y_dtype))
        return Q4_ERR_ENUM;
    const int sh = check_mx4(M, N, K);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(x, 16) || (x_dtype == Q4_MX4 && !aligned(x_scales, 4)) || !aligned(Wq, 16) || !aligned(w_scales, 4) ||
        !aligned(y, y_dtype == Q4_F32 ? 4 : 2))
        return Q4_ERR_ALIGN;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::mx4_workspace_bytes(x_dtype != Q4_MX4, M, N, K))
        return Q4_ERR_WORKSPACE;
    return hip_status(q4::launch_mx4_linear(x, x_dtype == Q4_MX4 ? -1 : elem_kind(x_dtype), (const uint8_t *)x_scales,
                                            (const uint8_t *)Wq, (const uint8_t *)w_scales, y, elem_kind(y_dtype), M, N,
                                            K, workspace, (hipStream_t)stream));
}

// Alignment of an element type's arrays where no wider one is asked for.
static uintptr_t elem_align(int dtype) { return dtype == Q4_F32 ? 4 : 2; }

static int check_norm(const q4_norm *n, q4::NormSide *out)
{
    *out = q4::NormSide{};
    if (!n || n->kind == Q4_NORM_NONE)
        return Q4_OK;
    if ((n->kind != Q4_NORM_RMS && n->kind != Q4_NORM_LAYER) || !is_float(n->dtype))
        return Q4_ERR_ENUM;
    if (!(n->eps >= 0.f && n->eps <= 3.4028235e38f))
        return Q4_ERR_SHAPE;
    if (!aligned(n->weight, elem_align(n->dtype)) || !aligned(n->bias, elem_align(n->dtype)))
        return Q4_ERR_ALIGN;
    *out = q4::NormSide{n->weight, n->bias, n->kind, elem_kind(n->dtype), n->eps};
    return Q4_OK;
}

int q4_block_norm(const void *y, int y_dtype, const q4_norm *post, const void *gate, int gate_dtype, int gate_form,
                  float scale, const void *residual, void *r, int r_dtype, const q4_norm *pre, void *h, int h_dtype,
                  void *h_scales, int M, int H, void *stream)
{
    if (!y || (!r && !h) || (gate_form != Q4_GATE_NONE && !gate) || (h && h_dtype == Q4_MX4 && !h_scales))
        return Q4_ERR_NULL;
    if (!is_float(y_dtype) || ((residual || r) && !is_float(r_dtype)) ||
        (h && !is_float(h_dtype) && h_dtype != Q4_MX4) || gate_form < Q4_GATE_NONE || gate_form > Q4_GATE_VALUE ||
        (gate_form != Q4_GATE_NONE && !is_float(gate_dtype)))
        return Q4_ERR_ENUM;
    const bool mx4 = h && h_dtype == Q4_MX4;
    if (M < 1 || H < 1 || M > (1 << 20) || H > Q4_NORM_MAX_H || (mx4 && H % 32 != 0))
        return Q4_ERR_SHAPE;
    if (!aligned(y, elem_align(y_dtype)) || ((residual || r) && (!aligned(residual, elem_align(r_dtype)) ||
                                                                 !aligned(r, elem_align(r_dtype)))) ||
        (gate_form != Q4_GATE_NONE && !aligned(gate, elem_align(gate_dtype))) ||
        (mx4 ? !aligned(h, 16) || !aligned(h_scales, 4) : h && !aligned(h, elem_align(h_dtype))))
        return Q4_ERR_ALIGN;
    q4::NormArgs a{};
    int st = check_norm(post, &a.post);
    if (st == Q4_OK)
        st = check_norm(pre, &a.pre);
    if (st != Q4_OK)
        return st;
    a.y = y;
    a.residual = residual;
    a.gate = gate;
    a.r = r;
    a.h = h;
    a.h_scales = mx4 ? (uint8_t *)h_scales : nullptr;
    a.y_type = elem_kind(y_dtype);
    a.r_type = elem_kind(r_dtype);
    a.h_type = mx4 ? 0 : elem_kind(h_dtype);
    a.gate_type = elem_kind(gate_dtype);
    a.gate_form = gate_form;
    a.scale = scale;
    a.M = M;
    a.H = H;
    return hip_status(q4::launch_block_norm(a, (hipStream_t)stream));
}

size_t q4_moe_route_workspace_bytes(int M, int E, int K)
{
    return check_moe(M, E, K, 1) == Q4_OK ? q4::moe_route_workspace_bytes(M, E, K) : 0;
}

int q4_moe_route(const void *x, int x_dtype, const void *router, int router_dtype, const float *bias, int *ids,
                 float *weights, int M, int E, int K, int topk, int renormalize, void *workspace,
                 size_t workspace_bytes, void *stream)
{
    if (!x || !router || !ids || !weights)
        return Q4_ERR_NULL;
    if ((x_dtype != Q4_F16 && x_dtype != Q4_BF16) || (router_dtype != x_dtype && router_dtype != Q4_F32))
        return Q4_ERR_ENUM;
    const int sh = check_moe(M, E, K, topk);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return Q4_ERR_ALIGN;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::moe_route_workspace_bytes(M, E, K))
        return Q4_ERR_WORKSPACE;
    return hip_status(q4::launch_moe_route(x, elem_kind(x_dtype), router, elem_kind(router_dtype), bias, ids, weights, M,
                                           E, K, topk, renormalize != 0, workspace, (hipStream_t)stream));
}

// (a row may name more experts than there are: ids repeat, or lie outside)
static int check_experts(int M, int E, int H, int I, int topk)
{
    const int sh = check_moe(M, E, H, 1);
    return sh != Q4_OK ? sh : check_moe(M, Q4_MOE_MAX_EXPERTS, I, topk);
}

size_t q4_moe_experts_workspace_bytes(int M, int H, int I, int topk)
{
    return check_experts(M, 1, H, I, topk) == Q4_OK ? q4::moe_workspace_bytes(M, H, I, topk) : 0;
}

int q4_moe_experts(const void *x, int x_dtype, const int *ids, const float *weights, const void *W13, const void *s13,
                   const void *W2, const void *s2, float *y, int M, int E, int H, int I, int topk, void *workspace,
                   size_t workspace_bytes, void *stream)
{
    if (!x || !ids || !weights || !W13 || !s13 || !W2 || !s2 || !y)
        return Q4_ERR_NULL;
    if (x_dtype != Q4_F16 && x_dtype != Q4_BF16)
        return Q4_ERR_ENUM;
    const int sh = check_experts(M, E, H, I, topk);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(x, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(W13, 16) || !aligned(s13, 8) ||
        !aligned(W2, 16) || !aligned(s2, 8) || !aligned(y, 4))
        return Q4_ERR_ALIGN;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::moe_workspace_bytes(M, H, I, topk))
        return Q4_ERR_WORKSPACE;
    return hip_status(q4::launch_moe_experts(x, x_dtype == Q4_BF16, ids, weights, (const uint8_t *)W13,
                                             (const uint16_t *)s13, (const uint8_t *)W2, (const uint16_t *)s2, y, M,
                                             topk, E, H, I, workspace, (hipStream_t)stream));
}

size_t q4_moe_layer_workspace_bytes(int M, int E, int H, int I, int topk)
{
    if (check_moe(M, E, H, topk) != Q4_OK || check_experts(M, E, H, I, topk) != Q4_OK)
        return 0;
    return q4::moe_layer_workspace_bytes(M, E, H, I, topk);
}

int q4_moe_layer(const void *x, int x_dtype, const void *router, int router_dtype, const float *bias, const void *W13,
                 const void *s13, const void *W2, const void *s2, float *y, int M, int E, int H, int I, int topk,
                 int renormalize, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!x || !router || !W13 || !s13 || !W2 || !s2 || !y)
        return Q4_ERR_NULL;
    if ((x_dtype != Q4_F16 && x_dtype != Q4_BF16) || (router_dtype != x_dtype && router_dtype != Q4_F32))
        return Q4_ERR_ENUM;
    int sh = check_moe(M, E, H, topk);
    if (sh == Q4_OK)
        sh = check_experts(M, E, H, I, topk);
    if (sh != Q4_OK)
        return sh;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(bias, 4) || !aligned(W13, 16) || !aligned(s13, 8) ||
        !aligned(W2, 16) || !aligned(s2, 8) || !aligned(y, 4))
        return Q4_ERR_ALIGN;
    if (workspace_bytes > 0 && !workspace)
        return Q4_ERR_WORKSPACE;
    if (workspace && !aligned(workspace, 256))
        return Q4_ERR_ALIGN;
    if (workspace_bytes < q4::moe_layer_workspace_bytes(M, E, H, I, topk))
        return Q4_ERR_WORKSPACE;
    return hip_status(q4::launch_moe_layer(x, elem_kind(x_dtype), router, elem_kind(router_dtype), bias,
                                           (const uint8_t *)W13, (const uint16_t *)s13, (const uint8_t *)W2,
                                           (const uint16_t *)s2, y, M, E, H, I, topk, renormalize != 0, workspace,
                                           (hipStream_t)stream));
}

}  // extern "C"
