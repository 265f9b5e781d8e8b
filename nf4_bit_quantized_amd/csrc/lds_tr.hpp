// MFMA operands whose contraction runs down the rows of an LDS tile
// (transposing LDS reads), and the swizzle that keeps them off each other's
// banks; shared by the kernels that form the adapter's gradients.
#pragma once

#include "common.hpp"

namespace qlora {
namespace ldstr {

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint16_t lds_u16_t;

// MFMA fragment from a row-major LDS tile [rows][ld] whose rows run along the
// contraction: lane l (i = l % 16) receives rows kb .. kb+7 of column c0 + i.
// ds_read_b64_tr_b16: within a 16-lane group, source lane s points at row
// kb + s/4, columns c0 + 4(s%4), and lane i receives rows kb..kb+3 of column c0+i.
__device__ __forceinline__ bf16x8_t tr_frag(const uint16_t* tile, int ld, int kb, int c0) {
  const int s = threadIdx.x & 15;
  const lds_u16_t* base = (const lds_u16_t*)tile;
  const int col = c0 + 4 * (s & 3);
  const int row = kb + (s >> 2);
  const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(base + row * ld + col));
  const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(base + (row + 4) * ld + col));
  const u16x8_t v = {(uint16_t)lo[0], (uint16_t)lo[1], (uint16_t)lo[2], (uint16_t)lo[3],
                     (uint16_t)hi[0], (uint16_t)hi[1], (uint16_t)hi[2], (uint16_t)hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// Row-major tiles read with transposing reads: the 16-byte piece p of row R
// is stored at piece p ^ tr_swz(R, pieces per row).  A transposing read (16
// lanes: four rows from a multiple of four, two adjacent pieces; the lanes of
// a 32-lane half take rows 8 further on) then touches each LDS bank at most
// once per 32 lanes (64 banks) and per 16 lanes (32 banks); with an
// unswizzled row of 64 bytes or more those rows fall on the same banks.  Row
// bit 2 is left out, so rows R and R + 4 (the two halves of a fragment) share
// the swizzle.  Widths of other piece counts keep the plain layout.
__device__ __forceinline__ int tr_swz(int row, int ppr) {
  const int b0 = row & 1, b1 = (row >> 1) & 1, b3 = (row >> 3) & 1;
  if (ppr == 4) return 2 * (b1 ^ b3);
  if (ppr == 8) return (2 * b0) ^ (4 * b1) ^ (2 * b3);
  if (ppr == 16 || ppr == 32 || ppr == 64) return (2 * b0) ^ (4 * b1) ^ (8 * b3);
  return 0;
}

// tr_frag from a tile stored with tr_swz (ld elements per row, a multiple of 8)
__device__ __forceinline__ bf16x8_t tr_frag_swz(const uint16_t* tile, int ld, int kb, int c0) {
  const int s = threadIdx.x & 15;
  const lds_u16_t* base = (const lds_u16_t*)tile;
  const int col = c0 + 4 * (s & 3);
  const int row = kb + (s >> 2);
  const int pcol = (((col >> 3) ^ tr_swz(row, ld >> 3)) << 3) | (col & 7);
  const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(base + row * ld + pcol));
  const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)(base + (row + 4) * ld + pcol));
  const u16x8_t v = {(uint16_t)lo[0], (uint16_t)lo[1], (uint16_t)lo[2], (uint16_t)lo[3],
                     (uint16_t)hi[0], (uint16_t)hi[1], (uint16_t)hi[2], (uint16_t)hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

}  // namespace ldstr
}  // namespace qlora
