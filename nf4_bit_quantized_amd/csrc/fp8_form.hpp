// The block scale and the codes of the 8-bit form (fp8.hip states the rule),
// shared by the kernels that write one.
#pragma once

#include "fp8.hpp"

namespace qlora {
namespace fp8 {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Bits of the largest |x|, what is not finite left out.
__device__ __forceinline__ uint32_t absmax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t u = __builtin_bit_cast(uint32_t, f[q]) & 0x7FFFFFFFu;
    m = u > m ? u : m;
  }
  if (m >= 0x7F800000u) {
    m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t u = __builtin_bit_cast(uint32_t, f[q]) & 0x7FFFFFFFu;
      m = u < 0x7F800000u && u > m ? u : m;
    }
  }
  return m;
}

__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  const int e = (int)((m + 0x1FFFFFu) >> 23) - 8;  // at most 247
  return (uint32_t)(e < 1 ? 1 : e);
}

// Eight codes; e in 1 .. 247, so the factor 2^(127 - e) is a normal float and
// the product is exact wherever the code is not zero.
__device__ __forceinline__ u32x2_t codes8(const float (&f)[8], uint32_t e) {
  const float k = __builtin_bit_cast(float, (254u - e) << 23);
  u32x2_t o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * k, f[4 * h + 1] * k, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * k, f[4 * h + 3] * k, w, true);
    o[h] = (uint32_t)w;
  }
  return o;
}

// The same for the two bf16 values of each of n dwords, as 16-bit integers: the
// bits of the largest finite |x|, as fp32.
template <class Dword>
__device__ __forceinline__ uint32_t absmax_bf16(int n, const Dword& x) {
  u16x2_t m = {0, 0};
#pragma unroll
  for (int q = 0; q < n; ++q) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, x(q) & 0x7FFF7FFFu));
  if (m[0] >= 0x7F80u || m[1] >= 0x7F80u) {
    m = u16x2_t{0, 0};
#pragma unroll
    for (int q = 0; q < n; ++q) {
      u16x2_t a = __builtin_bit_cast(u16x2_t, x(q) & 0x7FFF7FFFu);
      a[0] = a[0] < 0x7F80u ? a[0] : (uint16_t)0;
      a[1] = a[1] < 0x7F80u ? a[1] : (uint16_t)0;
      m = __builtin_elementwise_max(m, a);
    }
  }
  return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
}

// Eight codes of four dwords of bf16 values.  The instruction divides by the
// scale and rounds once, so its results are those of codes8 (the tests compare
// the two forms on every finite bf16 value, in blocks of neighbours, of twenty
// binades and of any sizes, and on what is not finite).
__device__ __forceinline__ u32x2_t codes8_bf16(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef short s16x2_t __attribute__((ext_vector_type(2)));
  const float k = __builtin_bit_cast(float, e << 23);
  const auto two = [&](uint32_t lo, uint32_t hi) {
    s16x2_t w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2_t, lo), k, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2_t, hi), k, true);
    return __builtin_bit_cast(uint32_t, w);
  };
  return u32x2_t{two(a, b), two(c, d)};
}

}  // namespace fp8
}  // namespace qlora
