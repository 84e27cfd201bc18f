// Block-scaled FP8 (E4M3 codes under fp32 scales) for gfx950: quantize and
// dequantize. A scale covers 1 x 128 elements of a row (activations) or a
// 128 x 128 tile (weights):
//   s    = fl32(amax / 448), 1 where amax = 0, NaN where an element is not finite
//   code = the E4M3 value nearest the exact quotient x / s, ties to the even
//          code, the sign copied; 0 under a NaN scale.
// The quotient of a bf16 x never reaches 464, where E4M3 would overflow: s is within
// half an fp32 step of amax / 448, at worst 2^-8 of it among the subnormals. (The
// fp32 values of norm_quantize.hip can be smaller than any bf16: fp8_encode.h.)
//
// Deciding the code without a division per element: x' rcp(s') is within 2^-21 of
// the quotient (x' and s' are scaled by 2^64 when s < 2^-60, so that neither the
// reciprocal overflows nor the product underflows), so the quotient lies between
// x' times rcp(s') (1 - 2^-20) and x' times rcp(s') (1 + 2^-20). Where both convert to the same code,
// that is the code. Otherwise one midpoint m of two neighbouring E4M3 values
// lies between them, and the sign of |x'| - m s', exact in one fma (m has 5
// bits), decides.
//
// Bound by HBM: 3.03 bytes an element, each read and written once.
#include "bf16.h"
#include "fp8_encode.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // 16-byte chunks per thread

__device__ __forceinline__ uint32_t chunk_absmax(u32x4 v) {
  const uint32_t m = 0x7FFF7FFFu;
  const u16x2 r = __builtin_elementwise_max(
      __builtin_elementwise_max(__builtin_bit_cast(u16x2, v.x & m), __builtin_bit_cast(u16x2, v.y & m)),
      __builtin_elementwise_max(__builtin_bit_cast(u16x2, v.z & m), __builtin_bit_cast(u16x2, v.w & m)));
  return r.x > r.y ? r.x : r.y;
}

// 1 x 128 blocks: the input is a flat array of 16-byte chunks (cols is a
// multiple of 128), 16 consecutive lanes (a DPP row) own a block.
__global__ __launch_bounds__(kThreads) void quant_fp8_rows_kernel(const u32x4* __restrict__ x,
                                                                  u32x2* __restrict__ codes,
                                                                  float* __restrict__ scales,
                                                                  int64_t nchunks) {
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  u32x4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; u++) {
    const int64_t c = base + u * kThreads;
    v[u] = c < nchunks ? __builtin_nontemporal_load(x + c) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int u = 0; u < kUnroll; u++) {
    const int64_t c = base + u * kThreads;
    const uint32_t m = fp8::row16_max(chunk_absmax(v[u]));
    const fp8::Scale s = fp8::scale_of(__builtin_bit_cast(float, m << 16));
    float e[8];
    unpack8(v[u], e);
    const uint2 q = fp8::encode8(e, s);
    if (c < nchunks) {
      // Plain stores: the GEMM that follows finds the codes in the caches.
      codes[c] = u32x2{q.x, q.y};
      if ((threadIdx.x & 15) == 0) scales[c >> 4] = s.value;
    }
  }
}

// 128 x 128 tiles: a workgroup of 8 waves takes 128 rows x 256 columns (two
// tiles; 28672 x 8192: 118.8 us = 5.9 TB/s, one tile 129, four 127), a load instruction two
// rows of them, and the tile stays in registers between its amax and its codes. The
// tiles' amax come from the waves' through LDS. Rows past the end belong to no
// tile; a tile at the end is shorter. Codes are not read again soon: non-temporal
// stores (plain ones: 125 us).
constexpr int W = 8;
__global__ __launch_bounds__(64 * W) void quant_fp8_tiles_kernel(
    const u32x4* __restrict__ x, u32x2* __restrict__ codes, float* __restrict__ scales, int64_t rows,
    int64_t cpr) {
  constexpr int kC = 4 * W, kTiles = W / 4;  // chunks of a row, tiles
  constexpr int kR = 64 / kC;                // rows of a load
  __shared__ uint32_t part[kTiles][W * kR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t across = (cpr + kC - 1) / kC, strip = blockIdx.x / across;  // strip: 128 rows
  const int tile = lane % kC / 16;
  const int64_t c = (int64_t)(blockIdx.x % across) * kC + lane % kC;         // chunk of the row
  const int64_t r0 = strip * 128 + wave * (8 * kR) + lane / kC;
  const bool in = c < cpr;
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; i++)
    v[i] = in && r0 + i * kR < rows ? __builtin_nontemporal_load(x + (r0 + i * kR) * cpr + c) : u32x4{0, 0, 0, 0};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint32_t a = chunk_absmax(v[i]);
    m = m > a ? m : a;
  }
  m = fp8::row16_max(m);
  if ((lane & 15) == 0) part[tile][wave * kR + lane / kC] = m;
  __syncthreads();
  static_assert(W * kR == 16, "a tile's partial maxima fill a DPP row");
  m = fp8::row16_max(part[tile][lane & 15]);
  const fp8::Scale s = fp8::scale_of(__builtin_bit_cast(float, m << 16));
  if (wave == 0 && lane < kC && (lane & 15) == 0 && in) scales[strip * (cpr / 16) + (c >> 4)] = s.value;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    float e[8];
    unpack8(v[i], e);
    const uint2 q = fp8::encode8(e, s);
    if (in && r0 + i * kR < rows) __builtin_nontemporal_store(u32x2{q.x, q.y}, codes + (r0 + i * kR) * cpr + c);
  }
}

// y = fl32(val(code) * s), 8 elements a thread and pass. tall: 128 x 128 tiles.
template <int OUT, bool TALL>
__global__ __launch_bounds__(kThreads) void dequant_fp8_kernel(const u32x2* __restrict__ codes,
                                                               const float* __restrict__ scales,
                                                               void* __restrict__ y, int64_t nchunks,
                                                               int64_t cpr) {
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < nchunks; c += (int64_t)gridDim.x * kThreads) {
    const float s = scales[TALL ? (c / cpr / 128) * (cpr / 16) + (c % cpr) / 16 : c >> 4];
    const u32x2 q = codes[c];
    float o[8];
    fp8::decode4(q.x, o);
    fp8::decode4(q.y, o + 4);
#pragma unroll
    for (int i = 0; i < 8; i++) o[i] *= s;
    if (OUT == kOutF32) {
      f32x4* p = (f32x4*)y + 2 * c;
      __builtin_nontemporal_store(f32x4{o[0], o[1], o[2], o[3]}, p);
      __builtin_nontemporal_store(f32x4{o[4], o[5], o[6], o[7]}, p + 1);
    } else {
      const u32x4 w = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
      __builtin_nontemporal_store(w, (u32x4*)y + c);
    }
  }
}

}  // namespace

hipError_t quant_fp8(int fmt, int64_t rows, int64_t cols, const void* x, void* codes, void* scales,
                     hipStream_t s) {
  const int64_t cpr = cols / 8;
  if (fmt == kFP8B128) {
    const int64_t n = rows * cpr, per = kThreads * kUnroll;
    return launch_kernel(&quant_fp8_rows_kernel, dim3((unsigned)((n + per - 1) / per)), kThreads, 0, s,
                         (const u32x4*)x, (u32x2*)codes, (float*)scales, n);
  }
  const dim3 grid((unsigned)((cpr + 4 * W - 1) / (4 * W) * ((rows + 127) / 128)));
  return launch_kernel(&quant_fp8_tiles_kernel, grid, 64 * W, 0, s, (const u32x4*)x, (u32x2*)codes,
                       (float*)scales, rows, cpr);
}

hipError_t dequant_fp8(int fmt, int64_t rows, int64_t cols, const void* codes, const void* scales,
                       int out_dtype, void* y, hipStream_t s) {
  const int64_t cpr = cols / 8, n = rows * cpr;
  // A pass per thread, but no more than a grid's 2^32 threads.
  const int64_t blocks = (n + kThreads - 1) / kThreads, most = (int64_t)1 << 23;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  const u32x2* q = (const u32x2*)codes;
  const float* sc = (const float*)scales;
  const bool tall = fmt == kFP8B128X128, f32 = out_dtype == kOutF32;
  if (tall && f32) return launch_kernel(&dequant_fp8_kernel<kOutF32, true>, grid, kThreads, 0, s, q, sc, y, n, cpr);
  if (tall) return launch_kernel(&dequant_fp8_kernel<kOutBF16, true>, grid, kThreads, 0, s, q, sc, y, n, cpr);
  if (f32) return launch_kernel(&dequant_fp8_kernel<kOutF32, false>, grid, kThreads, 0, s, q, sc, y, n, cpr);
  return launch_kernel(&dequant_fp8_kernel<kOutBF16, false>, grid, kThreads, 0, s, q, sc, y, n, cpr);
}

}  // namespace mx
