// Device helpers shared by the block-cooperative W4A4 kernels
// (gemm_w4a4_coop.hip, moe_w4a4.hip).  Internal; not part of the public ABI.
#pragma once

#include "qlin_internal.hpp"

namespace qlin {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ half2_t cvt2(uint32_t w, int sel) {
  switch (sel) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  }
}

// 8 codes -> 8 exact fp16 products with the group scale, packed for one store
__device__ __forceinline__ u32x4 dequant8(uint32_t w, half2_t s) {
  return u32x4{__builtin_bit_cast(uint32_t, cvt2(w, 0) * s),
               __builtin_bit_cast(uint32_t, cvt2(w, 1) * s),
               __builtin_bit_cast(uint32_t, cvt2(w, 2) * s),
               __builtin_bit_cast(uint32_t, cvt2(w, 3) * s)};
}

// E4M3 scale g (0..3) of a dword of four, as an fp16 pair: one packed
// conversion per two scales (exact: every E4M3 value is an fp16 value; an
// exhaustive GPU check of all byte pairs agreed), broadcast by the multiply
__device__ __forceinline__ half2_t scale_h2(uint32_t w4, int g) {
  const half2_t two = g < 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w4, 1.0f, false)
                            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w4, 1.0f, true);
  const _Float16 h = two[g & 1];
  return half2_t{h, h};
}

__device__ __forceinline__ uint32_t pick(const uint4& v, int d) {
  return d == 0 ? v.x : d == 1 ? v.y : d == 2 ? v.z : v.w;
}

}  // namespace
}  // namespace qlin
