// Internal launch interface of libmx (not part of the public ABI).
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <tuple>
#include <utility>

namespace mx {

// Launches kernel<<<grid, block, shmem, stream>>>(args...) through
// hipLaunchKernel and returns the status of that launch itself. (A status
// read back with hipGetLastError afterwards could instead be an error that
// an earlier HIP call of the caller left pending on this thread, and reading
// it would also clear the caller's error.) Arguments are converted to the
// kernel's parameter types first.
template <typename... P, typename... A, size_t... I>
inline hipError_t launch_impl(void (*kernel)(P...), dim3 grid, dim3 block, size_t shmem,
                              hipStream_t stream, std::index_sequence<I...>, A&&... args) {
  std::tuple<P...> params(static_cast<P>(std::forward<A>(args))...);
  void* argv[] = {(void*)&std::get<I>(params)...};
  return hipLaunchKernel((const void*)kernel, grid, block, argv, shmem, stream);
}

template <typename... P, typename... A>
inline hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t shmem,
                                hipStream_t stream, A&&... args) {
  static_assert(sizeof...(P) == sizeof...(A), "kernel argument count");
  return launch_impl(kernel, grid, block, shmem, stream, std::index_sequence_for<P...>{},
                     std::forward<A>(args)...);
}

// Returns from the enclosing launcher with the first failed launch's status.
#define MX_TRY(launch)                     \
  do {                                     \
    const hipError_t mx_e_ = (launch);     \
    if (mx_e_ != hipSuccess) return mx_e_; \
  } while (0)

// Format ids, kept equal to the public mx_format values.
enum : int { kBF16 = 0, kMXFP4 = 1, kMXFP8 = 2, kNVFP4 = 3, kMXFP8E5M2 = 4, kMXFP6 = 5, kMXFP4MBS = 6,
             kMXFP4MBS16 = 7, kFP8B128 = 8, kFP8B128X128 = 9 };
enum : int { kOutF32 = 0, kOutBF16 = 1 };

// ---- quantize.hip
// oas: MXFP4's overflow-aware scale rule; rot: 32-point Walsh-Hadamard rotation first.
// panel: codes and scales in the K-panel layout (panels of 256 elements for
// MXFP4, of 64 for MXFP8, E5M2 and E3M2; cols a multiple of that).
hipError_t quant_mx(int fmt, int64_t rows, int64_t cols, const void* x, void* codes,
                    void* scales, hipStream_t s, bool oas = false,
                    bool rot = false, bool panel = false);
// MXFP4 with static macro-block scaling over base blocks of `base` (16 or
// 32) elements: scales holds the E8M0 plane [rows][cols/base] followed by the
// macro mantissa plane [rows][cols/128].
hipError_t quant_mbs(int64_t rows, int64_t cols, const void* x, void* codes, void* scales,
                     hipStream_t s, int base);
size_t quant_nvfp4_workspace(int64_t rows, int64_t cols);
// panel: codes and scales in the K-panel layout with 64-element panels.
hipError_t quant_nvfp4(int64_t rows, int64_t cols, const void* x, void* codes, void* scales,
                       float* tensor_scale, void* workspace, hipStream_t s, bool panel = false);

// ---- dequantize.hip
hipError_t dequant(int fmt, int64_t rows, int64_t cols, const void* codes, const void* scales,
                   const float* tensor_scale, int out_dtype, void* y, hipStream_t s);

// ---- gemm_mx.hip (MXFP4 x MXFP4 on the FP4 scaled MFMA: the 256 x 256-tile
// kernel when it fits, else 128 x 128 tiles)
hipError_t gemm_mx(int64_t M, int64_t N, int64_t K, const void* a, const void* sa, const void* b,
                   const void* sb, int out_dtype, void* c, int64_t ldc, hipStream_t s);

// ---- gemm_mx.hip, MXFP4-MBS x MXFP4-MBS (128 x 128 tiles, any K % 128 = 0);
// sa / sb are the two-plane scale buffers.
hipError_t gemm_mbs_small(int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                          const void* b, const void* sb, int out_dtype, void* c, int64_t ldc,
                          hipStream_t s, int base);

// ---- gemm_mbs.hip (MXFP4-MBS x MXFP4-MBS over base blocks of `base` = 32 or
// 16 elements; 256 x 256 tiles when they fit, else gemm_mbs_small)
bool gemm_mbs_fits(int64_t M, int64_t N, int64_t K);
hipError_t gemm_mbs(int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                    const void* b, const void* sb, int out_dtype, void* c, int64_t ldc,
                    hipStream_t s, int base);

// ---- gemm_mxfp4.hip (MXFP4 x MXFP4, 256 x 256 tiles, register-staged
// pipeline); panel_a / panel_b: that operand in the K-panel layout (its
// rows * K / 2 below 2^31)
bool gemm_mxfp4_fits(int64_t M, int64_t N, int64_t K);
hipError_t gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                      const void* b, const void* sb, int out_dtype, void* c, int64_t ldc,
                      hipStream_t s, bool panel_a, bool panel_b);

// By expert (gemm_block's arguments), row layout.
hipError_t gemm_mxfp4_grouped(int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                              const void* b, const void* sb, const int32_t* offsets, int64_t groups,
                              int out_dtype, void* c, int64_t ldc, hipStream_t s);

// ---- pack.hip (codes and scales into the K-panel layout): `panels` panels,
// wb code bytes (a multiple of 16) and sb scale bytes (8, 4 or 2) per row
// and panel.
hipError_t pack_kpanel(int64_t rows, int64_t panels, int wb, int sb, const void* codes,
                       const void* scales, void* packed_codes, void* packed_scales, hipStream_t s);

// ---- gemm_bf16x.hip (MXFP8 x MXFP8 and NVFP4 x NVFP4, expanded exactly to bf16)
hipError_t gemm_bf16x(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                      const float* ta, const void* b, const void* sb, const float* tb,
                      int out_dtype, void* c, int64_t ldc, hipStream_t s);

// ---- gemm_bf16x_large.hip (256 x 256 or 224 x 256 tiles; MXFP8 / NVFP4 on the bf16 MFMA)
bool gemm_bf16x_large_fits(int fmt, int64_t M, int64_t N, int64_t K);
// panel: both operands in the K-panel layout (64-element panels).
hipError_t gemm_bf16x_large(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                            const float* ta, const void* b, const void* sb, const float* tb,
                            int out_dtype, void* c, int64_t ldc, hipStream_t s, bool panel = false);

// ---- fp8_block.hip: E4M3 codes under fp32 scales (kFP8B128: per 1 x 128,
// scales [rows][cols/128]; kFP8B128X128: per 128 x 128, [ceil(rows/128)][cols/128])
hipError_t quant_fp8(int fmt, int64_t rows, int64_t cols, const void* x, void* codes, void* scales,
                     hipStream_t s);
hipError_t dequant_fp8(int fmt, int64_t rows, int64_t cols, const void* codes, const void* scales,
                       int out_dtype, void* y, hipStream_t s);

// ---- gemm_block.hip: C = A B^T, dense (offsets null; FP8) or by expert (rows
// offsets[g] .. offsets[g+1]-1 against weight g of `groups`, offsets on the
// device). fmt: kMXFP4 (both operands) or kFP8B128 (B is kFP8B128X128).
bool gemm_block_fits(int64_t M, int64_t N, int64_t K, int64_t groups);
hipError_t gemm_block(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                      const void* b, const void* sb, const int32_t* offsets, int64_t groups,
                      int out_dtype, void* c, int64_t ldc, hipStream_t s);

// ---- gemm_fp8_large.hip (256 x 256 tiles, bf16 result; gemm_block's FP8 shapes)
hipError_t gemm_fp8_large(int64_t M, int64_t N, int64_t K, const void* a, const void* sa, const void* b,
                          const void* sb, const int32_t* offsets, int64_t groups, void* c, int64_t ldc,
                          hipStream_t s);

// ---- gemm_few_rows.hip (few rows of A, or few per expert: weights streamed
// once per 16 rows; gemm_block's shapes and arguments)
bool gemm_few_rows_fits(int64_t M, int64_t N, int64_t K, int64_t groups, int out_dtype);
hipError_t gemm_few_rows(int fmt, int64_t M, int64_t N, int64_t K, const void* a, const void* sa,
                         const void* b, const void* sb, const int32_t* offsets, int64_t groups,
                         int out_dtype, void* c, int64_t ldc, hipStream_t s);

// ---- norm_quantize.hip (kMXFP4, kMXFP8 or kFP8B128; cols at most kNormMaxCols;
// panel: elements per K panel of the codes and scales, 0 for the row layout)
constexpr int64_t kNormMaxCols = 32768;
hipError_t norm_quantize(int fmt, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                         const void* residual, int64_t ldr, const void* gate, int64_t gate_rows,
                         const void* post_weight, float alpha, const void* weight, float eps, void* h,
                         int64_t ldh, void* codes, void* scales, hipStream_t s, int panel);

// ---- gemm_w4a16.hip: the library's own scratch for mx_gemm_noalloc (the
// W4A16 split-K partials), a file-scope device array of this many bytes per
// GPU; noalloc_scratch returns its address on the current device (looked up
// once per device).
constexpr size_t kNoAllocScratchBytes = (size_t)8 << 20;
constexpr int kMaxDevices = 64;
hipError_t noalloc_scratch(void** ptr);

// ---- gemm_w4a16.hip (bf16 activations x MXFP4 weights)
size_t gemm_w4a16_workspace(int64_t M, int64_t N, int64_t K);
hipError_t gemm_w4a16(int64_t M, int64_t N, int64_t K, const void* a, const void* b,
                      const void* sb, int out_dtype, void* c, int64_t ldc, void* workspace,
                      hipStream_t s);

}  // namespace mx
