// C ABI of libmx: argument checks, dispatch to the gfx950 kernels, and error
// mapping. Every check runs before anything is enqueued; nothing here
// allocates, synchronizes or prints.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/mx.h"
#include "mx_internal.h"

namespace {

thread_local int g_last_hip_error = 0;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

bool is_quant_fmt(int f) {
  return f == MX_FMT_MXFP4 || f == MX_FMT_MXFP8 || f == MX_FMT_NVFP4 || f == MX_FMT_MXFP8_E5M2 ||
         f == MX_FMT_MXFP6_E3M2 || f == MX_FMT_MXFP4_MBS || f == MX_FMT_MXFP4_MBS16 ||
         f == MX_FMT_FP8_B128 || f == MX_FMT_FP8_B128X128 || f == MX_FMT_INT8;
}
bool is_mbs(int f) { return f == MX_FMT_MXFP4_MBS || f == MX_FMT_MXFP4_MBS16; }
bool is_fp8b(int f) { return f == MX_FMT_FP8_B128 || f == MX_FMT_FP8_B128X128; }
int block_of(int f) {
  if (f == MX_FMT_INT8) return 0;  // the whole row
  if (is_fp8b(f)) return 128;
  return (f == MX_FMT_NVFP4 || f == MX_FMT_MXFP4_MBS16) ? 16 : 32;
}
// fp32 scales need the alignment of a float, the others' bytes are read wide.
bool scales_aligned(int f, const void* p) { return is_fp8b(f) || f == MX_FMT_INT8 ? aligned4(p) : aligned16(p); }
// cols (and K) must be a multiple of this: the block, or the 128-element macro
// block of MXFP4-MBS and MXFP4-MBS16, or the 16 bytes of a load of INT8's rows.
int granule_of(int f) { return is_mbs(f) ? 128 : f == MX_FMT_INT8 ? 16 : block_of(f); }  // (the FP8 formats' block is 128)

// Elements per tensor stay below 2^40 and every GEMM extent below 2^30 so that
// the kernels' index arithmetic (int64 offsets, int extents) cannot overflow.
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxExtent = (int64_t)1 << 30;
constexpr int64_t kW4A16MaxK = 65536;
constexpr int64_t kMoeMaxWidth = (int64_t)1 << 20;  // hidden, inter and x's row stride of mx_moe
constexpr int64_t kMoeMaxWeight = (int64_t)1 << 30;  // hidden inter: 32-bit offsets in an expert's projection
constexpr int64_t kMaxGroups = 65535;  // experts of a grouped GEMM (a grid dimension)

mx_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MX_OK;
  g_last_hip_error = (int)e;
  return MX_ERR_HIP;
}

// Elements per K panel of a K-panel tensor: 256 for MXFP4 (one step of its
// GEMM), 64 for MXFP8, E5M2, E3M2 and NVFP4 (one stage of theirs).
int panel_width(int fmt) { return fmt == MX_FMT_MXFP4 ? 256 : 64; }

// Code bytes of a row of cols elements.
int64_t code_bytes(int fmt, int64_t cols) {
  if (fmt == MX_FMT_MXFP8 || fmt == MX_FMT_MXFP8_E5M2 || is_fp8b(fmt) || fmt == MX_FMT_INT8) return cols;
  if (fmt == MX_FMT_MXFP6_E3M2) return cols * 3 / 4;
  return cols / 2;
}

// Formats with a K-panel layout.
bool has_panel(int fmt) {
  return fmt == MX_FMT_MXFP4 || fmt == MX_FMT_MXFP8 || fmt == MX_FMT_MXFP8_E5M2 ||
         fmt == MX_FMT_MXFP6_E3M2 || fmt == MX_FMT_NVFP4;
}

// A K-panel tensor: whole panels, at most 65535 of them (a grid dimension of
// the panel quantizer), and 32-bit byte offsets.
bool panel_shape_ok(int fmt, int64_t rows, int64_t cols) {
  const int w = panel_width(fmt);
  return cols % w == 0 && cols / w <= 65535 && rows < ((int64_t)1 << 31) / code_bytes(fmt, cols);
}

// Common checks for a [rows][cols] quantized tensor.
mx_status check_tensor(int fmt, int block, int rnd, int64_t rows, int64_t cols) {
  if (!is_quant_fmt(fmt) || block != block_of(fmt)) return MX_ERR_UNSUPPORTED;
  if (rnd != MX_ROUND_RNE) return MX_ERR_UNSUPPORTED;
  if (rows <= 0 || cols <= 0 || cols % granule_of(fmt) != 0) return MX_ERR_INVALID_ARG;
  if (rows > kMaxElems / cols) return MX_ERR_INVALID_ARG;
  return MX_OK;
}

}  // namespace

extern "C" {

size_t mx_quantize_workspace_bytes(mx_format fmt, int64_t rows, int64_t cols) {
  if (fmt != MX_FMT_NVFP4 || rows <= 0 || cols <= 0) return 0;
  return mx::quant_nvfp4_workspace(rows, cols);
}

mx_status mx_quantize_layout(mx_format fmt, int block, mx_round rnd, int64_t rows, int64_t cols,
                             const void* x, void* codes, void* scales, float* tensor_scale,
                             void* workspace, size_t workspace_bytes, void* stream,
                             mx_layout layout) {
  mx_status st = check_tensor(fmt, block, rnd, rows, cols);
  if (st != MX_OK) return st;
  if (layout != MX_LAYOUT_ROWS && layout != MX_LAYOUT_KPANEL) return MX_ERR_UNSUPPORTED;
  const bool panel = layout == MX_LAYOUT_KPANEL;
  if (panel && !has_panel(fmt)) return MX_ERR_UNSUPPORTED;
  if (panel && !panel_shape_ok(fmt, rows, cols)) return MX_ERR_INVALID_ARG;
  if (!x || !codes || !scales) return MX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !scales_aligned(fmt, scales)) return MX_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (fmt == MX_FMT_NVFP4) {
    if (!tensor_scale || !aligned4(tensor_scale)) return MX_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace)) return MX_ERR_INVALID_ARG;
    if (workspace_bytes < mx::quant_nvfp4_workspace(rows, cols)) return MX_ERR_INVALID_ARG;
    return hip_status(mx::quant_nvfp4(rows, cols, x, codes, scales, tensor_scale, workspace, s, panel));
  }
  if (tensor_scale) return MX_ERR_INVALID_ARG;
  if (is_mbs(fmt)) return hip_status(mx::quant_mbs(rows, cols, x, codes, scales, s, block));
  if (fmt == MX_FMT_INT8) return hip_status(mx::quant_int8(rows, cols, x, codes, scales, s));
  if (is_fp8b(fmt)) return hip_status(mx::quant_fp8(fmt, rows, cols, x, codes, scales, s));
  return hip_status(mx::quant_mx(fmt, rows, cols, x, codes, scales, s, false, false, panel));
}

mx_status mx_quantize(mx_format fmt, int block, mx_round rnd, int64_t rows, int64_t cols,
                      const void* x, void* codes, void* scales, float* tensor_scale,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return mx_quantize_layout(fmt, block, rnd, rows, cols, x, codes, scales, tensor_scale, workspace,
                            workspace_bytes, stream, MX_LAYOUT_ROWS);
}

mx_status mx_quantize_ex(mx_format fmt, int block, mx_round rnd, mx_scale_rule rule,
                         mx_rotation rot, int64_t rows, int64_t cols, const void* x,
                         void* codes, void* scales, void* stream, mx_layout layout) {
  mx_status st = check_tensor(fmt, block, rnd, rows, cols);
  if (st != MX_OK) return st;
  if (layout != MX_LAYOUT_ROWS && layout != MX_LAYOUT_KPANEL) return MX_ERR_UNSUPPORTED;
  const bool panel = layout == MX_LAYOUT_KPANEL;
  if (fmt != MX_FMT_MXFP4 && fmt != MX_FMT_MXFP8) return MX_ERR_UNSUPPORTED;
  if (panel && !panel_shape_ok(fmt, rows, cols)) return MX_ERR_INVALID_ARG;
  if (rule != MX_SCALE_CEIL && !(rule == MX_SCALE_OAS && fmt == MX_FMT_MXFP4))
    return MX_ERR_UNSUPPORTED;
  if (rot != MX_ROTATE_NONE && rot != MX_ROTATE_WHT32) return MX_ERR_UNSUPPORTED;
  if (!x || !codes || !scales) return MX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MX_ERR_INVALID_ARG;
  return hip_status(mx::quant_mx(fmt, rows, cols, x, codes, scales, (hipStream_t)stream,
                                 rule == MX_SCALE_OAS, rot == MX_ROTATE_WHT32, panel));
}

mx_status mx_dequantize(mx_format fmt, int block, mx_round rnd, int64_t rows, int64_t cols,
                        const void* codes, const void* scales, const float* tensor_scale,
                        mx_dtype out_dtype, void* y, void* stream) {
  mx_status st = check_tensor(fmt, block, rnd, rows, cols);
  if (st != MX_OK) return st;
  if (out_dtype != MX_OUT_F32 && out_dtype != MX_OUT_BF16) return MX_ERR_UNSUPPORTED;
  if (!codes || !scales || !y) return MX_ERR_INVALID_ARG;
  if (!aligned16(codes) || !scales_aligned(fmt, scales) || !aligned16(y)) return MX_ERR_INVALID_ARG;
  if (fmt == MX_FMT_NVFP4) {
    if (!tensor_scale || !aligned4(tensor_scale)) return MX_ERR_INVALID_ARG;
  } else if (tensor_scale) {
    return MX_ERR_INVALID_ARG;
  }
  if (fmt == MX_FMT_INT8)
    return hip_status(mx::dequant_int8(rows, cols, codes, scales, out_dtype, y, (hipStream_t)stream));
  if (is_fp8b(fmt))
    return hip_status(mx::dequant_fp8(fmt, rows, cols, codes, scales, out_dtype, y, (hipStream_t)stream));
  return hip_status(mx::dequant(fmt, rows, cols, codes, scales, tensor_scale, out_dtype, y,
                                (hipStream_t)stream));
}

size_t mx_gemm_workspace_bytes(mx_format fmt_a, mx_format fmt_b, int64_t M, int64_t N, int64_t K) {
  if (fmt_a == MX_FMT_BF16 && fmt_b == MX_FMT_MXFP4 && M > 0 && N > 0 && K > 0 && K % 32 == 0 &&
      M <= kMaxExtent && N <= kMaxExtent && K <= kW4A16MaxK)
    return mx::gemm_w4a16_workspace(M, N, K);
  return 0;
}

}  // extern "C"

namespace {

// mx_gemm and mx_gemm_ex; panel_a / panel_b: that operand in the K-panel layout.
mx_status gemm_impl(mx_format fmt_a, mx_format fmt_b, int block, mx_round rnd, int64_t M, int64_t N,
                    int64_t K, const void* a, const void* a_scales, const float* a_ts,
                    const void* b, const void* b_scales, const float* b_ts, mx_dtype out_dtype,
                    void* c, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream,
                    bool panel_a, bool panel_b) {
  const bool w4a4 = fmt_a == MX_FMT_MXFP4 && fmt_b == MX_FMT_MXFP4 && block == 32;
  const bool w8a8 = fmt_a == MX_FMT_MXFP8 && fmt_b == MX_FMT_MXFP8 && block == 32;
  const bool nv = fmt_a == MX_FMT_NVFP4 && fmt_b == MX_FMT_NVFP4 && block == 16;
  const bool w4a16 = fmt_a == MX_FMT_BF16 && fmt_b == MX_FMT_MXFP4 && block == 32;
  const bool alt = fmt_a == fmt_b && block == 32 &&
                   (fmt_a == MX_FMT_MXFP8_E5M2 || fmt_a == MX_FMT_MXFP6_E3M2);
  const bool mbs = (fmt_a == MX_FMT_MXFP4_MBS && fmt_b == MX_FMT_MXFP4_MBS && block == 32) ||
                   (fmt_a == MX_FMT_MXFP4_MBS16 && fmt_b == MX_FMT_MXFP4_MBS16 && block == 16);
  const bool fp8b = fmt_a == MX_FMT_FP8_B128 && fmt_b == MX_FMT_FP8_B128X128 && block == 128;
  const bool int8 = fmt_a == MX_FMT_INT8 && fmt_b == MX_FMT_INT8 && block == 0;
  if (!(w4a4 || w8a8 || nv || w4a16 || alt || mbs || fp8b || int8)) return MX_ERR_UNSUPPORTED;
  // K-panel operands: the MXFP4 pair (either operand or both), or both
  // operands of the pairs on the 16-bit MFMAs.
  if ((panel_a || panel_b) && !w4a4 && !((w8a8 || nv || alt) && panel_a && panel_b))
    return MX_ERR_UNSUPPORTED;
  if (rnd != MX_ROUND_RNE) return MX_ERR_UNSUPPORTED;
  if (out_dtype != MX_OUT_F32 && out_dtype != MX_OUT_BF16) return MX_ERR_UNSUPPORTED;
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent)
    return MX_ERR_INVALID_ARG;
  // K is a whole number of 32-element groups for every path (NVFP4 included:
  // its 16-blocks are staged in pairs) but INT8's, of 16-byte loads.
  if (K % (int8 ? 16 : 32) != 0 || (int8 && K > mx::kInt8MaxK) || ((mbs || fp8b) && K % 128 != 0)) return MX_ERR_INVALID_ARG;
  if (ldc < N) return MX_ERR_INVALID_ARG;
  if ((fp8b || int8) && !mx::gemm_block_fits(M, N, K, 0)) return MX_ERR_INVALID_ARG;
  // Row tiles run along gridDim.y (at most 65535): 128 rows per tile for the
  // W4A4/W8A8 kernels, 16 for W4A16.
  if (M > (w4a16 ? 16 : 128) * (int64_t)65535) return MX_ERR_INVALID_ARG;
  // W4A16: at most 32 K-splits of 2048, so that each output's fp32 chain (33
  // roundings in a split, then the fixed-order sum of the splits) stays within
  // 64 steps, the accumulation bound of mx.h.
  if (w4a16 && K > kW4A16MaxK) return MX_ERR_INVALID_ARG;
  if (!a || !b || !b_scales || !c) return MX_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !scales_aligned(fmt_b, b_scales) || !aligned16(c))
    return MX_ERR_INVALID_ARG;
  if (w4a16) {
    if (a_scales || a_ts || b_ts) return MX_ERR_INVALID_ARG;
  } else {
    if (!a_scales || !scales_aligned(fmt_a, a_scales)) return MX_ERR_INVALID_ARG;
  }
  if (nv) {
    if (!a_ts || !b_ts || !aligned4(a_ts) || !aligned4(b_ts)) return MX_ERR_INVALID_ARG;
  } else if (a_ts || b_ts) {
    return MX_ERR_INVALID_ARG;
  }
  const size_t need = mx_gemm_workspace_bytes(fmt_a, fmt_b, M, N, K);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return MX_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (panel_a || panel_b) {
    if ((panel_a && !panel_shape_ok(fmt_a, M, K)) || (panel_b && !panel_shape_ok(fmt_b, N, K)))
      return MX_ERR_INVALID_ARG;
    if (!w4a4) {
      // The large-tile kernel of the 16-bit MFMAs reads K-panel operands.
      if (!mx::gemm_bf16x_large_fits(fmt_a, M, N, K)) return MX_ERR_INVALID_ARG;
      return hip_status(mx::gemm_bf16x_large(fmt_a, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                                             out_dtype, c, ldc, s, true));
    }
    // Only the 256 x 256-tile kernel reads K-panel MXFP4 operands.
    if (!mx::gemm_mxfp4_fits(M, N, K)) return MX_ERR_INVALID_ARG;
    return hip_status(mx::gemm_mxfp4(M, N, K, a, a_scales, b, b_scales, out_dtype, c, ldc, s,
                                     panel_a, panel_b));
  }
  if (w4a4)
    return hip_status(mx::gemm_mx(M, N, K, a, a_scales, b, b_scales, out_dtype, c, ldc, s));
  if (fp8b)
    return hip_status(mx::gemm_block(fmt_a, M, N, K, a, a_scales, b, b_scales, nullptr, 0, out_dtype, c, ldc, s));
  if (int8)
    return hip_status(mx::gemm_int8(M, N, K, a, a_scales, b, b_scales, nullptr, 0, out_dtype, c, ldc, s));
  if (mbs)
    return hip_status(mx::gemm_mbs(M, N, K, a, a_scales, b, b_scales, out_dtype, c, ldc, s, block));
  if (w8a8 || nv)
    return hip_status(mx::gemm_bf16x(fmt_a, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                                     out_dtype, c, ldc, s));
  if (alt) {
    if (!mx::gemm_bf16x_large_fits(fmt_a, M, N, K)) return MX_ERR_INVALID_ARG;
    return hip_status(mx::gemm_bf16x_large(fmt_a, M, N, K, a, a_scales, nullptr, b, b_scales,
                                           nullptr, out_dtype, c, ldc, s));
  }
  return hip_status(mx::gemm_w4a16(M, N, K, a, b, b_scales, out_dtype, c, ldc, workspace, s));
}

// [p, p + n) and [q, q + m) share a byte.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + m && b < a + n;
}

}  // namespace

extern "C" {

mx_status mx_gemm(mx_format fmt_a, mx_format fmt_b, int block, mx_round rnd, int64_t M, int64_t N,
                  int64_t K, const void* a, const void* a_scales, const float* a_ts,
                  const void* b, const void* b_scales, const float* b_ts, mx_dtype out_dtype,
                  void* c, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream) {
  return gemm_impl(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                   out_dtype, c, ldc, workspace, workspace_bytes, stream, false, false);
}

mx_status mx_gemm_ex(mx_format fmt_a, mx_format fmt_b, int block, mx_round rnd, int64_t M,
                     int64_t N, int64_t K, const void* a, const void* a_scales, const float* a_ts,
                     const void* b, const void* b_scales, const float* b_ts, mx_dtype out_dtype,
                     void* c, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream,
                     mx_layout a_layout, mx_layout b_layout) {
  if (a_layout != MX_LAYOUT_ROWS && a_layout != MX_LAYOUT_KPANEL) return MX_ERR_UNSUPPORTED;
  if (b_layout != MX_LAYOUT_ROWS && b_layout != MX_LAYOUT_KPANEL) return MX_ERR_UNSUPPORTED;
  return gemm_impl(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                   out_dtype, c, ldc, workspace, workspace_bytes, stream,
                   a_layout == MX_LAYOUT_KPANEL, b_layout == MX_LAYOUT_KPANEL);
}

mx_status mx_gemm_noalloc(mx_format fmt_a, mx_format fmt_b, int block, mx_round rnd, int64_t M,
                          int64_t N, int64_t K, const void* a, const void* a_scales,
                          const float* a_ts, const void* b, const void* b_scales,
                          const float* b_ts, mx_dtype out_dtype, void* c, int64_t ldc,
                          void* stream) {
  const size_t need = mx_gemm_workspace_bytes(fmt_a, fmt_b, M, N, K);
  void* ws = nullptr;
  if (need > 0) {
    if (need > mx::kNoAllocScratchBytes) return MX_ERR_INVALID_ARG;
    const hipError_t e = mx::noalloc_scratch(&ws);
    if (e != hipSuccess) return hip_status(e);
  }
  return gemm_impl(fmt_a, fmt_b, block, rnd, M, N, K, a, a_scales, a_ts, b, b_scales, b_ts,
                   out_dtype, c, ldc, ws, need, stream, false, false);
}

mx_status mx_gemm_grouped(mx_format fmt_a, mx_format fmt_b, int block, mx_round rnd, int64_t groups,
                          int64_t M, int64_t N, int64_t K, const int32_t* offsets, const void* a,
                          const void* a_scales, const void* b, const void* b_scales,
                          mx_dtype out_dtype, void* c, int64_t ldc, void* stream) {
  const bool w4a4 = fmt_a == MX_FMT_MXFP4 && fmt_b == MX_FMT_MXFP4 && block == 32;
  const bool fp8b = fmt_a == MX_FMT_FP8_B128 && fmt_b == MX_FMT_FP8_B128X128 && block == 128;
  const bool int8 = fmt_a == MX_FMT_INT8 && fmt_b == MX_FMT_INT8 && block == 0;
  if (!(w4a4 || fp8b || int8)) return MX_ERR_UNSUPPORTED;
  if (rnd != MX_ROUND_RNE) return MX_ERR_UNSUPPORTED;
  if (out_dtype != MX_OUT_F32 && out_dtype != MX_OUT_BF16) return MX_ERR_UNSUPPORTED;
  if (M <= 0 || N <= 0 || K <= 0 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent)
    return MX_ERR_INVALID_ARG;
  if (groups <= 0 || groups > kMaxGroups || M > kMaxElems / K || groups * N > kMaxElems / K)
    return MX_ERR_INVALID_ARG;
  if (K % granule_of(fmt_a) != 0 || (int8 && K > mx::kInt8MaxK) || ldc < N) return MX_ERR_INVALID_ARG;
  if (!mx::gemm_block_fits(M, N, K, groups)) return MX_ERR_INVALID_ARG;
  if (!offsets || !aligned4(offsets)) return MX_ERR_INVALID_ARG;
  if (!a || !a_scales || !b || !b_scales || !c) return MX_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c)) return MX_ERR_INVALID_ARG;
  if (!scales_aligned(fmt_a, a_scales) || !scales_aligned(fmt_b, b_scales)) return MX_ERR_INVALID_ARG;
  if (int8)
    return hip_status(mx::gemm_int8(M, N, K, a, a_scales, b, b_scales, offsets, groups, out_dtype, c, ldc,
                                    (hipStream_t)stream));
  return hip_status(mx::gemm_block(fmt_a, M, N, K, a, a_scales, b, b_scales, offsets, groups, out_dtype,
                                   c, ldc, (hipStream_t)stream));
}

size_t mx_moe_workspace_bytes(int64_t tokens, int64_t top, int64_t experts, int64_t hidden, int64_t inter) {
  if (tokens <= 0 || top <= 0 || experts <= 0 || hidden <= 0 || inter <= 0) return 0;
  if (tokens > mx::kMoeMaxTokens || top > mx::kMoeMaxTop || experts > mx::kMoeMaxExperts) return 0;
  if (hidden > kMoeMaxWidth || inter > kMoeMaxWidth) return 0;
  return mx::moe_workspace(tokens, top, experts, hidden, inter);
}

mx_status mx_moe(mx_format fmt, int block, mx_round rnd, int64_t tokens, int64_t top, int64_t experts,
                 int64_t hidden, int64_t inter, const void* x, int64_t ldx, const int32_t* ids,
                 const float* weights, const void* up, const void* up_scales, const void* down,
                 const void* down_scales, mx_dtype out_dtype, void* y, int64_t ldy, void* workspace,
                 size_t workspace_bytes, void* stream) {
  if ((fmt != MX_FMT_MXFP4 && fmt != MX_FMT_FP8_B128X128 && fmt != MX_FMT_INT8) || block != block_of(fmt)) return MX_ERR_UNSUPPORTED;
  if (rnd != MX_ROUND_RNE) return MX_ERR_UNSUPPORTED;
  if (out_dtype != MX_OUT_F32 && out_dtype != MX_OUT_BF16) return MX_ERR_UNSUPPORTED;
  // (0: a size or a limit)
  const size_t need = mx_moe_workspace_bytes(tokens, top, experts, hidden, inter);
  if (need == 0 || hidden % granule_of(fmt) != 0 || inter % granule_of(fmt) != 0) return MX_ERR_INVALID_ARG;
  if (hidden > kMoeMaxWeight / inter) return MX_ERR_INVALID_ARG;
  // Rows of x are read 16 bytes at a time at 32-bit offsets, those of y written 4 elements at a time.
  if (ldx < hidden || ldx % 8 != 0 || ldx > kMoeMaxWidth || ldy < hidden || ldy % 4 != 0 || ldy > kMaxExtent) return MX_ERR_INVALID_ARG;
  if (!x || !ids || !weights || !up || !up_scales || !down || !down_scales || !y || !workspace) return MX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned4(ids) || !aligned4(weights) || !aligned16(up) || !aligned16(down) || !aligned16(y)) return MX_ERR_INVALID_ARG;
  if (!scales_aligned(fmt, up_scales) || !scales_aligned(fmt, down_scales)) return MX_ERR_INVALID_ARG;
  if (!aligned16(workspace) || workspace_bytes < need) return MX_ERR_INVALID_ARG;
  return hip_status(mx::moe(fmt, tokens, top, experts, hidden, inter, x, ldx, ids, weights, up, up_scales, down, down_scales,
                            out_dtype, y, ldy, workspace, (hipStream_t)stream));
}

mx_status mx_norm_quantize(mx_format fmt, int block, mx_round rnd, int64_t rows, int64_t cols,
                           const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           const void* gate, int64_t gate_rows, const void* post_weight, float alpha,
                           const void* weight, float eps, void* h, int64_t ldh, void* codes,
                           void* scales, void* stream, mx_layout layout) {
  if (fmt != MX_FMT_MXFP4 && fmt != MX_FMT_MXFP8 && fmt != MX_FMT_FP8_B128) return MX_ERR_UNSUPPORTED;
  mx_status st = check_tensor(fmt, block, rnd, rows, cols);
  if (st != MX_OK) return st;
  if (layout != MX_LAYOUT_ROWS && layout != MX_LAYOUT_KPANEL) return MX_ERR_UNSUPPORTED;
  const bool panel = layout == MX_LAYOUT_KPANEL;
  if (panel && !has_panel(fmt)) return MX_ERR_UNSUPPORTED;
  if (panel && !panel_shape_ok(fmt, rows, cols)) return MX_ERR_INVALID_ARG;
  if (cols > mx::kNormMaxCols) return MX_ERR_INVALID_ARG;
  // Rows are read and written 16 bytes at a time.
  if (ldx < cols || ldx % 8 != 0 || rows > kMaxElems / ldx) return MX_ERR_INVALID_ARG;
  if (residual && (ldr < cols || ldr % 8 != 0 || rows > kMaxElems / ldr)) return MX_ERR_INVALID_ARG;
  if (h && (ldh < cols || ldh % 8 != 0 || rows > kMaxElems / ldh)) return MX_ERR_INVALID_ARG;
  if (gate && gate_rows <= 0) return MX_ERR_INVALID_ARG;
  // (negated, so that NaN fails too)
  if (!(eps >= 0.0f && eps < HUGE_VALF) || !(alpha > -HUGE_VALF && alpha < HUGE_VALF)) return MX_ERR_INVALID_ARG;
  if (!x || !codes || !scales) return MX_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !scales_aligned(fmt, scales)) return MX_ERR_INVALID_ARG;
  if (!aligned16(residual) || !aligned16(gate) || !aligned16(post_weight) || !aligned16(weight) || !aligned16(h))
    return MX_ERR_INVALID_ARG;
  return hip_status(mx::norm_quantize(fmt, rows, cols, x, ldx, residual, ldr, gate, gate_rows, post_weight,
                                      alpha, weight, eps, h, ldh, codes, scales, (hipStream_t)stream,
                                      panel ? panel_width(fmt) : 0));
}

mx_status mx_pack(mx_format fmt, int block, int64_t rows, int64_t cols, const void* codes,
                  const void* scales, void* packed_codes, void* packed_scales, void* stream) {
  if (!has_panel(fmt) || block != block_of(fmt)) return MX_ERR_UNSUPPORTED;
  if (rows <= 0 || cols <= 0 || !panel_shape_ok(fmt, rows, cols)) return MX_ERR_INVALID_ARG;
  if (!codes || !scales || !packed_codes || !packed_scales) return MX_ERR_INVALID_ARG;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(packed_codes) || !aligned16(packed_scales))
    return MX_ERR_INVALID_ARG;
  const size_t cb = (size_t)rows * (size_t)code_bytes(fmt, cols),
               sb = (size_t)rows * (size_t)(cols / block);
  if (overlap(codes, cb, packed_codes, cb) || overlap(codes, cb, packed_scales, sb) ||
      overlap(scales, sb, packed_codes, cb) || overlap(scales, sb, packed_scales, sb))
    return MX_ERR_INVALID_ARG;
  const int w = panel_width(fmt);
  return hip_status(mx::pack_kpanel(rows, cols / w, (int)code_bytes(fmt, w), w / block, codes, scales,
                                    packed_codes, packed_scales, (hipStream_t)stream));
}

int mx_last_hip_error(void) { return g_last_hip_error; }

const char* mx_status_string(mx_status s) {
  switch (s) {
    case MX_OK: return "MX_OK";
    case MX_ERR_INVALID_ARG: return "MX_ERR_INVALID_ARG";
    case MX_ERR_UNSUPPORTED: return "MX_ERR_UNSUPPORTED";
    case MX_ERR_HIP: return "MX_ERR_HIP";
  }
  return "MX_ERR_UNKNOWN";
}

}  // extern "C"
