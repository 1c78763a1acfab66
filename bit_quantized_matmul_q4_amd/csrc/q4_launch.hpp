// q4_launch.hpp -- host-side launchers exported by q4_kernels.hip to the C
// ABI layer (q4_api.cpp).  Arguments are already validated by the caller.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace q4 {

// Multi-row matrix-vector kernel: any M (rows are processed 16 at a time).
hipError_t launch_gemv(const void *x, bool bf16, const uint8_t *wq, const uint16_t *scales,
                       float *y, int M, int N, int K, hipStream_t stream);

// One matrix of a group that shares x, M and K.
struct GroupItem {
    const uint8_t *wq;
    const uint16_t *scales;
    float *y;
    int N;
};

// The group (1..8 matrices) in one launch of the matrix-vector kernel: the
// segment form where it takes K, else the split form.  Returns false,
// launching nothing, for a group whose total width calls for the streaming
// form (then *err is untouched); else the launch status in *err.
bool launch_gemv_grouped(const void *x, bool bf16, const GroupItem *items, int count, int M, int K,
                         hipStream_t stream, hipError_t *err);

// LDS-staged matrix-matrix kernel.  workspace may be NULL (no split of K
// across workgroups); otherwise it holds workspace_bytes bytes.
hipError_t launch_gemm(const void *x, bool bf16, const uint8_t *wq, const uint16_t *scales,
                       float *y, int M, int N, int K, void *workspace, size_t workspace_bytes,
                       hipStream_t stream);

// Bytes of workspace the matrix-matrix kernel can use for this shape.
size_t gemm_workspace_bytes(int M, int N, int K);

// The library's fixed per-device scratch buffer (for the entry point that
// allocates nothing): its size, and its device address on the current device
// (looked up once per device).
constexpr size_t kScratchBytes = size_t(4) << 20;
hipError_t scratch_buffer(void **ptr);

// Canonical codes ([N][K] one per byte, or nibble rows [N][K/2]) and
// scales [N][K/32] -> the tiled layout.
hipError_t launch_pack(const uint8_t *codes, bool nibbles, const uint16_t *scales_in, uint8_t *wq,
                       uint16_t *scales_out, int N, int K, hipStream_t stream);

// Dense weights [N][K] (kind 0 binary16, 1 bfloat16, 2 binary32) ->
// canonical codes [N][K] and binary16 scales [N][K/32].
hipError_t launch_quantize(const void *w, int kind, uint8_t *codes, uint16_t *scales, int N, int K,
                           hipStream_t stream);

// The matrix product in 8-bit integers (q4_int8.hip).  Element kinds: 0
// binary16, 1 bfloat16, 2 binary32.
// Dense rows [rows][K] -> codes (canonical [rows][K] or packed) and scales.
hipError_t launch_int8_quantize(const void *x, int kind, int8_t *codes, bool packed, float *scales, int rows, int K,
                                hipStream_t stream);
// Canonical codes [rows][K] -> packed.
hipError_t launch_int8_pack(const int8_t *codes, int8_t *packed, int rows, int K, hipStream_t stream);
size_t int8_packed_bytes(int rows, int K);
// y = x . W^T; x_kind -1: x is packed codes with x_scales; 0 or 1: dense
// rows, quantized into the workspace (which holds int8_workspace_bytes).
hipError_t launch_int8_linear(const void *x, int x_kind, const float *x_scales, const int8_t *wq, const float *w_scales,
                              void *y, int y_kind, int M, int N, int K, void *workspace, hipStream_t stream);
size_t int8_workspace_bytes(bool dense, int M, int N, int K);

// The expert layer (q4_moe.hip).
hipError_t launch_moe_route(const void *x, int x_kind, const void *router, int r_kind, const float *bias, int *ids,
                            float *weights, int M, int E, int K, int topk, int renormalize, void *workspace,
                            hipStream_t stream);
size_t moe_route_workspace_bytes(int M, int E, int K);
hipError_t launch_moe_experts(const void *x, bool bf16, const int *ids, const float *weights, const uint8_t *w13,
                              const uint16_t *s13, const uint8_t *w2, const uint16_t *s2, float *y, int M, int topk,
                              int E, int H, int I, void *workspace, hipStream_t stream);
size_t moe_workspace_bytes(int M, int H, int I, int topk);
hipError_t launch_moe_layer(const void *x, int x_kind, const void *router, int r_kind, const float *bias,
                            const uint8_t *w13, const uint16_t *s13, const uint8_t *w2, const uint16_t *s2, float *y,
                            int M, int E, int H, int I, int topk, int renormalize, void *workspace, hipStream_t stream);
size_t moe_layer_workspace_bytes(int M, int E, int H, int I, int topk);

// The microscaled 4-bit form and its product (q4_mx4.hip).  Element kinds as
// above.
// Dense rows [rows][K] -> codes and scale bytes (canonical or packed).
hipError_t launch_mx4_quantize(const void *x, int kind, uint8_t *codes, uint8_t *scales, bool packed, int rows, int K,
                               hipStream_t stream);
// Canonical -> packed; packed -> values [rows][K].
hipError_t launch_mx4_pack(const uint8_t *codes, const uint8_t *scales, uint8_t *packed, uint8_t *tiles, int rows,
                           int K, hipStream_t stream);
hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, void *y, int kind, int rows, int K,
                                 hipStream_t stream);
size_t mx4_code_bytes(int rows, int K);
size_t mx4_scale_bytes(int rows, int K);
// y = x . W^T; x_kind -1: x is packed codes with x_scales; 0 or 1: dense
// rows, quantized in the call (the workspace holds mx4_workspace_bytes).
hipError_t launch_mx4_linear(const void *x, int x_kind, const uint8_t *x_scales, const uint8_t *wq, const uint8_t *ws,
                             void *y, int y_kind, int M, int N, int K, void *workspace, hipStream_t stream);
size_t mx4_workspace_bytes(bool dense, int M, int N, int K);

// The norms around a block (q4_norm.hip).  Types: element kinds as above.
struct NormSide {
    const void *weight, *bias;  // [H] of `type`, either may be NULL
    int kind;                   // 0 none, 1 rms, 2 layer
    int type;
    float eps;
};
struct NormArgs {
    const void *y, *residual, *gate;  // residual may be NULL
    void *r, *h;                      // either may be NULL
    uint8_t *h_scales;                // not NULL: h is packed microscaled 4-bit rows
    NormSide post, pre;
    int y_type, r_type, h_type, gate_type;
    int gate_form;  // 0 none, 1 [H], 2 [M], 3 [M][H]
    float scale;
    int M, H;
};
hipError_t launch_block_norm(const NormArgs &args, hipStream_t stream);

// Sizes of the tiled layout.
size_t packed_code_bytes(int N, int K);
size_t packed_scale_bytes(int N, int K);

}  // namespace q4
