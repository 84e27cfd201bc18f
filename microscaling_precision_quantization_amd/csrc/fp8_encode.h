// E4M3 codes under an fp32 scale: the scale from a block's amax, and codes
// that are nearest to the exact quotient x / s (see fp8_block.hip); and codes back
// to values.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace mx {
namespace fp8 {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Max of v over each DPP row of 16 lanes, in every lane of the row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  uint32_t o;
#define MX_ROR(n)                                                                         \
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xF, 0xF, false);       \
  v = v > o ? v : o;
  MX_ROR(8) MX_ROR(4) MX_ROR(2) MX_ROR(1)
#undef MX_ROR
  return v;
}

// A block's scale: the stored value, and what encode8 works with: the scale
// times `lift` (2^64 for s < 2^-60, else 1), and its reciprocal a little
// lowered and raised. An amax whose quotient rounds to 0 (up to 1.75 * 2^-142) is
// stored under 1, as 0 is: its codes are zeros.
struct Scale {
  float value, lifted, lift, down, up;
  bool finite;
};

__device__ __forceinline__ Scale scale_of(float amax) {
  Scale s;
  s.finite = __builtin_bit_cast(uint32_t, amax) < 0x7F800000u;
  float v = amax / 448.0f;
  if (v == 0.0f) v = 1.0f;
  s.value = s.finite ? v : __builtin_nanf("");
  s.lift = v < 0x1p-60f ? 0x1p64f : 1.0f;
  s.lifted = v * s.lift;
  const float inv = __builtin_amdgcn_rcpf(s.lifted);
  s.down = inv * (1.0f - 0x1p-20f);
  s.up = inv * (1.0f + 0x1p-20f);
  return s;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int q = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, q, true);
}

__device__ __forceinline__ void decode4(uint32_t q, float* o) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, true);
  o[0] = a.x; o[1] = a.y; o[2] = b.x; o[3] = b.y;
}

// 8 E4M3 codes as bf16.
__device__ __forceinline__ bf16x8 expand8(int lo, int hi) {
  u32x4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, true));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, false));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, true));
  return __builtin_bit_cast(bf16x8, o);
}

// The code between two neighbouring candidates lo < hi (magnitudes' codes, or
// the same): the exact comparison of |x'| with their midpoint times s'.
__device__ __forceinline__ uint32_t settle(uint32_t lo, uint32_t hi, float x, const Scale& s) {
  if (lo == hi) return lo;
  const uint32_t a = lo & 0x7Fu;
  const float m = 0.5f * (__builtin_amdgcn_cvt_f32_fp8((int)a, 0) + __builtin_amdgcn_cvt_f32_fp8((int)(a + 1), 0));
  const float d = __builtin_fmaf(-m, s.lifted, __builtin_fabsf(x));
  const uint32_t up = d > 0.0f || (d == 0.0f && (a & 1)) ? 1u : 0u;
  return lo + up;
}

// Codes of 8 elements of a block with scale s (zero if it is not finite).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const Scale& s) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i++) y[i] = x[i];
  if (s.lift != 1.0f) {
    // Among the fp32 subnormals a scale can be so coarse that quotients pass 464,
    // where the conversion would give NaN: saturate.
    const float most = 448.0f * s.lifted;
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = __builtin_amdgcn_fmed3f(y[i] * s.lift, -most, most);
  }
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const float* v = y + 4 * h;
    lo[h] = pack4(v[0] * s.down, v[1] * s.down, v[2] * s.down, v[3] * s.down);
    hi[h] = pack4(v[0] * s.up, v[1] * s.up, v[2] * s.up, v[3] * s.up);
  }
  if (((lo[0] ^ hi[0]) | (lo[1] ^ hi[1])) != 0) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      uint32_t q = 0;
#pragma unroll
      for (int i = 0; i < 4; i++)
        q |= settle((lo[h] >> (8 * i)) & 0xFFu, (hi[h] >> (8 * i)) & 0xFFu, y[4 * h + i], s) << (8 * i);
      lo[h] = q;
    }
  }
  return s.finite ? uint2{lo[0], lo[1]} : uint2{0u, 0u};
}

}  // namespace fp8
}  // namespace mx
