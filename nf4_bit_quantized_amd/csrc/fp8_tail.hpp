// Operands of the adapter's rank-r term where it runs as a tail of a product
// of 8-bit forms: eight consecutive columns c .. c+7 of the 2r hi/lo columns.
#pragma once

#include "fp8.hpp"

namespace qlora {

// of feature row n
__device__ __forceinline__ bf16x8_t tail_weight(const Fp8Params& p, int64_t n, int64_t rows, int c) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (n < rows) {
    if (p.bt_pair) {
      v = *reinterpret_cast<const uint4*>(p.Bt + n * p.ldh + c);
    } else if (c < 2 * p.r) {
      v = *reinterpret_cast<const uint4*>(p.Bt + n * p.r + (c < p.r ? c : c - p.r));
    }
  }
  return __builtin_bit_cast(bf16x8_t, v);
}

// of token t
__device__ __forceinline__ bf16x8_t tail_token(const Fp8Params& p, int64_t t, int c) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (t < p.T) v = *reinterpret_cast<const uint4*>(p.At + t * p.ldh + c);
  return __builtin_bit_cast(bf16x8_t, v);
}

}  // namespace qlora
