// The scales of an 8-bit integer product: C = sum * s_A * s_B, the sum an int32.
// The scales' significands and exponents are multiplied and added apart, so that
// no intermediate product leaves fp32's range where C is in it: the sum's
// conversion, the significands' product and the result round once each.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace mx {
namespace int8 {

struct Scale {
  float m;  // in [1/2, 1); 0, Inf and NaN as they are
  int e;
};

__device__ __forceinline__ Scale split(float s) {
  return {__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}

__device__ __forceinline__ float apply(int sum, const Scale& a, const Scale& b) {
  return __builtin_ldexpf((float)sum * (a.m * b.m), a.e + b.e);
}

}  // namespace int8
}  // namespace mx
