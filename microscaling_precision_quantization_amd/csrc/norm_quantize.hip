// The norms between two blocks of a transformer and the quantizer after them,
// in one pass (rows of x are the first block's output):
//   y = x, or post_weight * x * rsqrt(mean(x^2) + eps)
//   h = residual + alpha * gate * y                (kept as bf16, if asked for)
//   n = weight * h * rsqrt(mean(h^2) + eps)
//   codes, scales = quantize(n)
// Everything between the bf16 inputs and the codes is fp32 in registers: the
// second norm reads h before its rounding to bf16, and the quantizer n before
// any, so the codes are nearer to the formula's than through two bf16
// tensors. Scales follow mx_quantize's rule, evaluated on the fp32 amax.
//
// A workgroup of T threads owns a row (up to 8 CH T elements, CH 16-byte chunks a
// thread, lane after lane), so both sums stay on chip and each input is read
// once: the kernel is bound by HBM. Weights and gate stay in registers over a
// workgroup's rows.
#include "bf16.h"
#include "fp8_encode.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Sum over the workgroup, the same bits in every thread. `part`: LDS that no
// earlier sum still reads.
template <int T>
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
  if (T == 64) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < T / 64; w++) s += part[w];
  return s;
}

struct NormArgs {
  const uint16_t *x, *residual, *gate, *post, *weight;
  uint16_t* h;
  uint8_t *codes, *scales;
  int64_t rows, ldx, ldr, ldh, gate_rows;
  int cols;
  float alpha, eps;
  int panel;  // elements per K panel, 0: row layout
};

template <int FMT, int T, int CH>
__global__ __launch_bounds__(T) void norm_quantize_kernel(NormArgs p) {
  __shared__ float part[4][16];
  const int tid = threadIdx.x;
  const int chunks = p.cols / 8;
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  auto chunk_of = [&](const uint16_t* v, int i) __attribute__((always_inline)) {
    const int c = i * T + tid;
    return v && c < chunks ? ((const u32x4*)v)[c] : ones;
  };
  // Rows of up to 4 chunks a thread have no VGPRs for them: the weights come from the
  // caches for every row, and no row is loaded ahead.
  constexpr bool kKeep = CH < 4;
  u32x4 w[CH], pw[CH], gt[CH];
#pragma unroll
  for (int i = 0; i < CH && kKeep; i++) {
    w[i] = chunk_of(p.weight, i);
    pw[i] = chunk_of(p.post, i);
    gt[i] = ones;
  }
  int64_t gate_at = -1;
  const float inv = 1.0f / (float)p.cols;
  int slot = 0;
  // The next row's inputs are loaded while a row is computed. (x and residual of
  // a row are read before h, which may be the same memory, is written for it.)
  u32x4 nx[CH], nr[CH];
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int c = i * T + tid;
      const bool in = c < chunks && row < p.rows;
      nx[i] = in ? __builtin_nontemporal_load((const u32x4*)(p.x + row * p.ldx) + c) : u32x4{0, 0, 0, 0};
      nr[i] = p.residual && in ? __builtin_nontemporal_load((const u32x4*)(p.residual + row * p.ldr) + c) : u32x4{0, 0, 0, 0};
    }
  };
  if (kKeep) fetch(blockIdx.x);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, slot ^= 2) {
    if (!kKeep) fetch(row);
    u32x4 vr[CH];
    float h[CH][8];
#pragma unroll
    for (int i = 0; i < CH; i++) {
      unpack8(nx[i], h[i]);
      vr[i] = nr[i];
    }
    if (kKeep) fetch(row + gridDim.x);
    const uint16_t* gate = p.gate ? p.gate + row / p.gate_rows * p.cols : nullptr;
    if (kKeep && gate && row / p.gate_rows != gate_at) {
      gate_at = row / p.gate_rows;
#pragma unroll
      for (int i = 0; i < CH; i++) gt[i] = chunk_of(gate, i);
    }
    float ry = p.alpha;  // what the products x post_weight gate are multiplied by
    if (p.post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; i++)
#pragma unroll
        for (int e = 0; e < 8; e++) ss = __builtin_fmaf(h[i][e], h[i][e], ss);
      ry = p.alpha / sqrtf(block_sum<T>(ss, part[slot]) * inv + p.eps);
    }
    // x post_weight gate has at most 24 significant bits and is exact, so h
    // rounds once per element.
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
      float f[8], q[8], r[8];
      unpack8(kKeep ? gt[i] : chunk_of(gate, i), f);
      unpack8(kKeep ? pw[i] : chunk_of(p.post, i), q);
      unpack8(vr[i], r);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        h[i][e] = __builtin_fmaf(h[i][e] * q[e] * f[e], ry, r[e]);
        ss = __builtin_fmaf(h[i][e], h[i][e], ss);
      }
    }
    if (p.h) {
#pragma unroll
      for (int i = 0; i < CH; i++) {
        const int c = i * T + tid;
        if (c >= chunks) continue;
        const u32x4 v = {pack_bf16x2(h[i][0], h[i][1]), pack_bf16x2(h[i][2], h[i][3]), pack_bf16x2(h[i][4], h[i][5]),
                         pack_bf16x2(h[i][6], h[i][7])};
        u32x4* dst = (u32x4*)(p.h + row * p.ldh) + c;
        __builtin_nontemporal_store(v, dst);
      }
    }
    const float rs = 1.0f / sqrtf(block_sum<T>(ss, part[slot + 1]) * inv + p.eps);
#pragma unroll
    for (int i = 0; i < CH; i++) {
      const int c = i * T + tid;
      float f[8], n[8];
      unpack8(kKeep ? w[i] : chunk_of(p.weight, i), f);
      uint32_t m = 0;  // amax as bits: a larger magnitude has larger bits
#pragma unroll
      for (int e = 0; e < 8; e++) {
        n[e] = h[i][e] * f[e] * rs;
        m = umax(m, __builtin_bit_cast(uint32_t, n[e]) & 0x7FFFFFFFu);
      }
      // Where this chunk's codes go, in elements from the tensor's start.
      int64_t at = row * p.cols + c * 8;
      if (p.panel) at = ((int64_t)(c * 8 / p.panel) * p.rows + row) * p.panel + c * 8 % p.panel;
      if constexpr (FMT == kFP8B128) {
        m = fp8::row16_max(m);
        const fp8::Scale s = fp8::scale_of(__builtin_bit_cast(float, m));
        const uint2 q = fp8::encode8(n, s);
        if (c < chunks) {
          *(u32x2*)(p.codes + at) = u32x2{q.x, q.y};
          if ((tid & 15) == 0) ((float*)p.scales)[at / 128] = s.value;
        }
      } else {
        m = umax(m, dpp<0xB1>(m));
        m = umax(m, dpp<0x4E>(m));
        // E = ceil(log2(amax / emax)) + 127, emax = 1.5 * 2^2 or 1.75 * 2^8.
        const int ea = (int)(m >> 23), ma = (int)(m & 0x7FFFFFu);
        int e = FMT == kMXFP4 ? ea - 2 + (ma > 0x400000) : ea - 8 + (ma > 0x600000);
        e = e < 0 ? 0 : e;
        const bool finite = m < 0x7F800000u;
        const float scale = __builtin_bit_cast(float, e == 0 ? 0x00400000u : (uint32_t)e << 23);
        if (FMT == kMXFP4) {
          uint32_t q = 0;
          q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, n[0], n[1], scale, 0);
          q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, n[2], n[3], scale, 1);
          q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, n[4], n[5], scale, 2);
          q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, n[6], n[7], scale, 3);
          if (c < chunks) *(uint32_t*)(p.codes + at / 2) = finite ? q : 0u;
        } else {
          i16x2 lo = {0, 0}, hi = {0, 0};
          lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, n[0], n[1], scale, false);
          lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, n[2], n[3], scale, true);
          hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, n[4], n[5], scale, false);
          hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, n[6], n[7], scale, true);
          const u32x2 q = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
          if (c < chunks) *(u32x2*)(p.codes + at) = finite ? q : u32x2{0, 0};
        }
        if (c < chunks && (tid & 3) == 0) p.scales[at / 32] = finite ? (uint8_t)e : (uint8_t)255;
      }
    }
  }
}

template <int FMT>
hipError_t launch(const NormArgs& p, hipStream_t s) {
  // Rows at a time: as many workgroups as the chip holds at 2048 threads a
  // CU, so that a workgroup keeps its weights over several rows.
  const int c = p.cols;
  const int64_t t = c <= 512 ? 64 : c <= 4096 ? 256 : c <= 8192 ? 512 : 1024;
  const int64_t most = 256 * (2048 / t);
  const dim3 grid((unsigned)(p.rows < most ? p.rows : most));
  if (c <= 512) return launch_kernel(&norm_quantize_kernel<FMT, 64, 1>, grid, 64, 0, s, p);
  if (c <= 2048) return launch_kernel(&norm_quantize_kernel<FMT, 256, 1>, grid, 256, 0, s, p);
  if (c <= 4096) return launch_kernel(&norm_quantize_kernel<FMT, 256, 2>, grid, 256, 0, s, p);
  if (c <= 8192) return launch_kernel(&norm_quantize_kernel<FMT, 512, 2>, grid, 512, 0, s, p);
  if (c <= 16384) return launch_kernel(&norm_quantize_kernel<FMT, 1024, 2>, grid, 1024, 0, s, p);
  return launch_kernel(&norm_quantize_kernel<FMT, 1024, 4>, grid, 1024, 0, s, p);
}

}  // namespace

hipError_t norm_quantize(int fmt, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                         const void* residual, int64_t ldr, const void* gate, int64_t gate_rows,
                         const void* post_weight, float alpha, const void* weight, float eps, void* h,
                         int64_t ldh, void* codes, void* scales, hipStream_t s, int panel) {
  const NormArgs p{(const uint16_t*)x, (const uint16_t*)residual, (const uint16_t*)gate,
                   (const uint16_t*)post_weight, (const uint16_t*)weight, (uint16_t*)h, (uint8_t*)codes,
                   (uint8_t*)scales, rows, ldx, ldr, ldh, gate_rows, (int)cols, alpha, eps, panel};
  if (fmt == kMXFP4) return launch<kMXFP4>(p, s);
  if (fmt == kMXFP8) return launch<kMXFP8>(p, s);
  return launch<kFP8B128>(p, s);
}

}  // namespace mx
