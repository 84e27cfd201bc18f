// 8-bit integers under one fp32 scale per row (a token of the activations, an
// output channel of a weight): quantize and dequantize.
//   s    = fl32(amax / 127) over the row, 1 where amax = 0, NaN where an element is not finite
//   code = the integer nearest the exact quotient x / s, ties to even; 0 under a NaN scale.
//
// Deciding the code with one fma an element. With A = amax, x / s differs from
// t = 127 x / A by s's rounding only, a factor within 2^-24 of 1 (normal s). x and A have 8
// significant bits each, so t either is a border h of two codes (an odd multiple of 1/2,
// at most 8 bits), or 254 x and 2 h A are different integers of at most 16 bits (up to a
// power of two): then t is at least 2^-16 of itself away from h. So x times 1 / s,
// lowered or raised by 2^-19 (more than the errors of the reciprocal and of s together, 2^-22),
// is on t's side of every border that t is not on, and where t is on one, the direction
// decides: down where s was rounded up (x / s is then below t), up where s was rounded
// down, as the sign of fma(s, 127, -A) says. Where s is exact, A's 8 bits are 127 times s's, s
// is a power of two and so is 1 / s: no lowering or raising, and ties are exact.
// fma(x, that, 1.5 * 2^23) rounds the exact product to an integer, ties to even,
// whose two's complement is the sum's low byte.
// A scale below 2^-100 (whose reciprocal may overflow, and whose rounding among the
// subnormals is coarser) takes the quotient in 64 bits: borders and x / s are then
// at least 2^-32 apart, or equal. No quotient reaches 127.5: s is within half an
// fp32 step of amax / 127, at worst 2^-10 of it.
//
// Bound by HBM: 3 bytes an element, each read and written once. A row stays in
// registers between its amax and its codes. Measured in us: 28672 x 8192 117 (6.0 TB/s), 8192 x 8192
// 34, 1024 x 8192 5.8. With non-temporal stores of the codes 110, 33 and 6.1, but the product of
// these with 4096 columns, which then finds them in no cache, takes 30, 3 and 2.5 more.
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
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // of 256 threads: 2^31, half of what a launch may have; each takes further rows

__device__ __forceinline__ uint32_t chunk_absmax(u32x4 v) {
  const uint32_t m = 0x7FFF7FFFu;
  const u16x2 r = __builtin_elementwise_max(
      __builtin_elementwise_max(__builtin_bit_cast(u16x2, v.x & m), __builtin_bit_cast(u16x2, v.y & m)),
      __builtin_elementwise_max(__builtin_bit_cast(u16x2, v.z & m), __builtin_bit_cast(u16x2, v.w & m)));
  return r.x > r.y ? r.x : r.y;
}

// Max over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = fp8::row16_max(v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * i);
    m = m > o ? m : o;
  }
  return m;
}

struct Scale {
  float value, s, inv;  // as stored; finite; what encode8 multiplies by
  bool finite;
};

__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
  Scale r;
  const float a = __builtin_bit_cast(float, amax_bits << 16);
  r.finite = amax_bits < 0x7F80u;
  r.s = a / 127.0f;
  if (r.s == 0.0f) r.s = 1.0f;
  r.value = r.finite ? r.s : __builtin_nanf("");
  const float up = __builtin_fmaf(r.s, 127.0f, -a);  // > 0: s was rounded up (amax = 0: any)
  r.inv = 1.0f / r.s * (up > 0.0f ? 1.0f - 0x1p-19f : up < 0.0f ? 1.0f + 0x1p-19f : 1.0f);
  return r;
}

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  // (v_perm: selectors 0..3 are bytes of the second operand, 4..7 of the first.)
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
  return lo | hi;
}

__device__ __forceinline__ u32x2 encode8(u32x4 v, const Scale& s) {
  float x[8];
  unpack8(v, x);
  uint32_t q[8];
  if (s.s >= 0x1p-100f) {
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = __builtin_bit_cast(uint32_t, __builtin_fmaf(x[i], s.inv, 12582912.0f));
  } else {
    for (int i = 0; i < 8; i++) q[i] = (uint32_t)(int)__builtin_rint((double)x[i] / (double)s.s);
  }
  const u32x2 r = {low_bytes(q[0], q[1], q[2], q[3]), low_bytes(q[4], q[5], q[6], q[7])};
  return s.finite ? r : u32x2{0, 0};
}

// LANES lanes (a wave or the workgroup) a row, of at most 8 LANES U elements: cpr
// chunks of 8.
template <int LANES, int U>
__global__ __launch_bounds__(kThreads) void quant_int8_kernel(const u32x4* __restrict__ x, u32x2* __restrict__ codes,
                                                              float* __restrict__ scales, int64_t rows, int cpr) {
  constexpr int kRows = kThreads / LANES;
  __shared__ uint32_t part[4];
  const int lane = threadIdx.x % LANES;
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < rows; row0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = row0 + threadIdx.x / LANES;
    const bool in = row < rows;
    u32x4 v[U];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int c = u * LANES + lane;
      v[u] = in && c < cpr ? __builtin_nontemporal_load(x + row * cpr + c) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t a = chunk_absmax(v[u]);
      m = m > a ? m : a;
    }
    m = wave_max(m);
    if (LANES > 64) {
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; w++) m = m > part[w] ? m : part[w];
      __syncthreads();
    }
    const Scale s = scale_of(m);
    if (in && lane == 0) scales[row] = s.value;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int c = u * LANES + lane;
      const u32x2 q = encode8(v[u], s);
      if (in && c < cpr) codes[row * cpr + c] = q;
    }
  }
}

// Longer rows: read twice, the second time from the caches, with one load on its way a thread: 8192 x 28672 184 us, where
// 28672 x 8192 takes 104.
__global__ __launch_bounds__(kThreads) void quant_int8_long_kernel(const u32x4* __restrict__ x, u32x2* __restrict__ codes,
                                                                   float* __restrict__ scales, int64_t rows, int64_t cpr) {
  __shared__ uint32_t part[4];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    uint32_t m = 0;
    for (int64_t c = threadIdx.x; c < cpr; c += kThreads) {
      const uint32_t a = chunk_absmax(x[row * cpr + c]);
      m = m > a ? m : a;
    }
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; w++) m = m > part[w] ? m : part[w];
    __syncthreads();
    const Scale s = scale_of(m);
    if (threadIdx.x == 0) scales[row] = s.value;
    for (int64_t c = threadIdx.x; c < cpr; c += kThreads) codes[row * cpr + c] = encode8(x[row * cpr + c], s);
  }
}

// y = fl32(code * s), 8 elements a thread and pass. 8192 x 8192 to bf16 31 us (5 TB/s and more: HBM), to fp32 102 (3.3 TB/s):
// there each of a thread's two stores leaves out every other 16 bytes of the lines that the wave's cover.
template <int OUT>
__global__ __launch_bounds__(kThreads) void dequant_int8_kernel(const u32x2* __restrict__ codes,
                                                                const float* __restrict__ scales,
                                                                void* __restrict__ y, int64_t nchunks, int64_t cpr) {
  for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < nchunks; c += (int64_t)gridDim.x * kThreads) {
    const float s = scales[c / cpr];
    const u32x2 q = codes[c];
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; i++) o[i] = (float)(int8_t)(q[i / 4] >> (8 * (i % 4))) * s;
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

template <int LANES, int U>
hipError_t launch_rows(int64_t rows, int64_t cpr, const void* x, void* codes, void* scales, hipStream_t s) {
  const int64_t per = kThreads / LANES, n = (rows + per - 1) / per;
  return launch_kernel(&quant_int8_kernel<LANES, U>, dim3((unsigned)(n < kMaxBlocks ? n : kMaxBlocks - 1)), kThreads, 0, s,
                       (const u32x4*)x, (u32x2*)codes, (float*)scales, rows, (int)cpr);
}

}  // namespace

hipError_t quant_int8(int64_t rows, int64_t cols, const void* x, void* codes, void* scales, hipStream_t s) {
  const int64_t cpr = cols / 8;
  if (cpr <= 64) return launch_rows<64, 1>(rows, cpr, x, codes, scales, s);
  if (cpr <= 128) return launch_rows<64, 2>(rows, cpr, x, codes, scales, s);
  if (cpr <= 256) return launch_rows<64, 4>(rows, cpr, x, codes, scales, s);
  if (cpr <= 512) return launch_rows<256, 2>(rows, cpr, x, codes, scales, s);
  if (cpr <= 1024) return launch_rows<256, 4>(rows, cpr, x, codes, scales, s);
  if (cpr <= 2048) return launch_rows<256, 8>(rows, cpr, x, codes, scales, s);
  return launch_kernel(&quant_int8_long_kernel, dim3((unsigned)(rows < kMaxBlocks ? rows : kMaxBlocks - 1)), kThreads, 0, s,
                       (const u32x4*)x, (u32x2*)codes, (float*)scales, rows, cpr);
}

hipError_t dequant_int8(int64_t rows, int64_t cols, const void* codes, const void* scales, int out_dtype, void* y,
                        hipStream_t s) {
  const int64_t cpr = cols / 8, n = rows * cpr, blocks = (n + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks - 1));
  if (out_dtype == kOutF32)
    return launch_kernel(&dequant_int8_kernel<kOutF32>, grid, kThreads, 0, s, (const u32x2*)codes, (const float*)scales, y, n, cpr);
  return launch_kernel(&dequant_int8_kernel<kOutBF16>, grid, kThreads, 0, s, (const u32x2*)codes, (const float*)scales, y, n, cpr);
}

}  // namespace mx
