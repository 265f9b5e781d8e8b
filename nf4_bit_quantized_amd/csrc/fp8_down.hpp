// U = X A^T over the 8-bit form of X: the tile that a workgroup forms beside the
// weight's stream in the few-token product (fp8_gemm.hip), and what it shares
// with the kernel of its own for more tokens (fp8_adapter.hip).
#pragma once

#include "fp8.hpp"

namespace qlora {
namespace fp8 {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// Eight codes (two dwords) restored: exact, save below bf16's subnormal steps
// and from 2^128 on, which is an infinity.
__device__ __forceinline__ u32x4_t restore8(uint32_t a, uint32_t b, float k) {
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, k, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, k, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, k, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, k, true))};
}

// red[w][t][j] = sum over the chunks c_begin + w, + NW, ... of 128 positions, of
// X[t0 + t][k] A[j0 + j][k], t, j < 16, by wave w of NW.  Fragments come straight
// from global memory: lane l of token row l % 16 takes the 32 codes 32 (l / 16) ..
// +31 of a chunk, which are its share of four MFMAs; four chunks' loads go out
// before the first is multiplied.  Loads of a row past the end, and of the missing
// half of a last chunk, repeat others: the sums of the one are never used, the
// codes of the other made zero.
template <int NW, int LD>
__device__ __forceinline__ void down_tile(const Fp8DownParams& p, int64_t t0, int j0, int c_begin, int c_end, int wave,
                                          float (*red)[16][LD]) {
  constexpr int DEPTH = 4;
  const int lane = threadIdx.x & 63;
  const int i = lane & 15, g = lane >> 4;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int64_t t = t0 + i < p.T ? t0 + i : p.T - 1;
  const int j = j0 + i < p.r ? j0 + i : p.r - 1;
  const uint8_t* xrow = p.X + t * p.K;
  const uint8_t* srow = p.Xs + t * fp8_scale_ld(p.K);
  const uint16_t* arow = p.A + (int64_t)j * p.K;
  for (int ch0 = c_begin + wave; ch0 < c_end; ch0 += DEPTH * NW) {
    u32x4_t x[DEPTH][2], a[DEPTH][4];
    uint32_t sb[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int ch = ch0 + d * NW < c_end ? ch0 + d * NW : ch0;
      const int64_t k = (int64_t)ch * 128 + 32 * g < p.K ? (int64_t)ch * 128 + 32 * g : 0;
      sb[d] = srow[ch];
#pragma unroll
      for (int q = 0; q < 2; ++q) x[d][q] = reinterpret_cast<const u32x4_t*>(xrow + k)[q];
#pragma unroll
      for (int q = 0; q < 4; ++q) a[d][q] = reinterpret_cast<const u32x4_t*>(arow + k)[q];
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int ch = ch0 + d * NW;
      const uint32_t keep = ch < c_end && (int64_t)ch * 128 + 32 * g < p.K ? 0xFFFFFFFFu : 0u;
      const float k = scale_of(sb[d]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const u32x4_t v = restore8(x[d][q >> 1][2 * (q & 1)] & keep, x[d][q >> 1][2 * (q & 1) + 1] & keep, k);
        acc = mfma16(__builtin_bit_cast(bf16x8_t, v),
                     __builtin_bit_cast(bf16x8_t, keep ? a[d][q] : u32x4_t{0u, 0u, 0u, 0u}), acc);
      }
    }
  }
  // lane l, value v: token 4 (l/16) + v, column l % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][4 * g + v][i] = acc[v];
}

}  // namespace fp8
}  // namespace qlora
