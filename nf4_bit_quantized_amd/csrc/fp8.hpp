// The 8-bit form of a matrix (e4m3 codes, one power-of-two scale per block of
// 1 x 128 or 128 x 128) and the kernels on it; see fp8.hip for the format.
#pragma once

#include "common.hpp"

namespace qlora {

constexpr int kFp8Block = 128;

// Bytes of one row of scales: one per block of 128 columns, in whole dwords.
__host__ __device__ inline int64_t fp8_scale_ld(int64_t cols) { return (cols + 511) / 512 * 4; }
inline int64_t fp8_scale_rows(int64_t rows, int block_rows) { return (rows + block_rows - 1) / block_rows; }

// M [rows][cols] (format kWeight*) -> codes, scales; block_rows 1 or 128, cols a multiple of 64.
hipError_t launch_fp8_quantize(const void* M, int format, int64_t rows, int64_t cols, int block_rows, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream);
// codes, scales -> bf16 [rows][cols]
hipError_t launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                 int block_rows, uint16_t* out, hipStream_t stream);

// C[t][n] = bf16( sum_k X[t][k] W[n][k] + sum_c At[t][c] Bt[n][c] )        (dx == 0)
// C[t][k] = bf16( sum_n X[t][n] W[n][k] + sum_c At[t][c] Bt[k][c] )        (dx == 1)
// X is the 8-bit form by rows (contraction contiguous), W [Nw][Kw] the 8-bit
// form by 128 x 128 blocks.  The tail runs over the 2r hi/lo columns of At.
struct Fp8Params {
  const uint8_t* X;
  const uint8_t* Xs;
  const uint8_t* W;
  const uint8_t* Ws;
  int64_t T, Nw, Kw;
  int32_t dx;
  int32_t r;           // 0: no tail
  const uint16_t* At;  // bf16 [T][ldh]: hi columns 0..r-1, lo columns r..2r-1, zeros to ldh
  int64_t ldh;         // a multiple of 64
  const uint16_t* Bt;  // bt_pair == 0: B [rows][r], r % 8 == 0; 1: [rows][ldh] (the pair operand)
  int32_t bt_pair;
  uint16_t* C;
  float* part;         // partial sums, fp8_product_part_bytes
  size_t part_bytes;
  // at most kFp8FewT tokens and r > 0: the rank-r term comes from these instead
  // of from At and Bt, and the forward's U is formed by the product's own launch
  float s;
  const uint16_t* A;   // forward: bf16 [r][Kw]
  const uint16_t* M;   // forward: B [Nw][r]; dx: A [r][Kw]
  const float* G;      // dx: fp32 [T][r]
  float* U;            // forward: receives U, or null
};
// The most tokens for which the product is a stream of the weight with the
// rank-r term in the pass behind it.  Forward, this way against U's own kernel
// and the tiles of plan_product: 4096 x 4096, r = 16: 21 us against 23 at 128
// tokens, 21 against 24 at 160; 8192 x 8192, r = 64: 34 and 36, 38.5 and 40;
// 11008 x 4096, r = 16: 26 and 27.5, 29 and 28.  Larger weights cross earlier:
// 28672 x 8192, r = 64: 72 and 77 at 64 tokens, 84 and 79 at 96, 93 and 80 at
// 128; 8192 x 28672: 69 and 72.5, 83 and 81, 86 and 81.  Whole backward passes
// cross between 128 and 160 tokens too (8192 x 8192: 53 and 54, 60 and 59); of
// 28672 x 8192 they are within 3% up to 96 tokens, 118 and 101 at 128.
constexpr int64_t kFp8FewT = 128;
size_t fp8_product_part_bytes(int64_t T, int64_t Nw, int64_t Kw, int dx, int r);
hipError_t launch_fp8_product(const Fp8Params& p, hipStream_t stream);

// The pair operand of a tail: out [rows][ldh] = (V | V | 0), V [rows][r] being
// B itself (transposed == 0: B [rows][r]) or A's transpose (1: A [r][rows]).
hipError_t launch_fp8_pair(const uint16_t* M, int64_t rows, int r, int64_t ldh, int transposed, uint16_t* out,
                           hipStream_t stream);

// U = X A^T from the 8-bit form of X: U [T][r] fp32 (optional) and the hi/lo
// pair of s*U into Us [T][ldh] (optional), zero-padded.
struct Fp8DownParams {
  const uint8_t* X;
  const uint8_t* Xs;
  const uint16_t* A;  // bf16 [r][K]
  int64_t T, K;
  int32_t r;
  float s;
  float* U;
  uint16_t* Us;
  int64_t ldh;
  float* part;
  size_t part_bytes;
};
size_t fp8_down_part_bytes(int64_t T, int64_t K, int r);
hipError_t launch_fp8_down(const Fp8DownParams& p, hipStream_t stream);

// G = dY B and the 8-bit form of dY in one pass over it: G [T][r] fp32, the
// hi/lo pair of s*G into Gs [T][ldh], zero-padded.  Where fp8_form_ok.
struct Fp8FormParams {
  const uint16_t* dY;  // bf16 [T][N]
  const uint16_t* B;   // bf16 [N][r]
  int64_t T, N;
  int32_t r;
  float s;
  uint8_t* codes;      // null: G alone
  uint8_t* scales;
  float* G;
  uint16_t* Gs;
  int64_t ldh;
  float* part;
  size_t part_bytes;
};
bool fp8_form_ok(int r);
size_t fp8_form_part_bytes(int64_t T, int64_t N, int r);
hipError_t launch_fp8_form(const Fp8FormParams& p, hipStream_t stream);

// The adapter's gradients: dA[j][k] = s sum_t G[t][j] X[t][k] over the 8-bit
// form of X, dB[n][j] = s sum_t dY[t][n] U[t][j]; G, U fp32 [T][r].
struct Fp8GradParams {
  const uint8_t* X;
  const uint8_t* Xs;
  const uint16_t* dY;  // bf16 [T][N]
  const float* G;
  const float* U;
  int64_t T, K, N;
  int32_t r;
  float s;
  float* dA;
  float* dB;
  int32_t accumulate;
  float* part;
  size_t part_bytes;
};
size_t fp8_grad_part_bytes(int64_t T, int64_t K, int64_t N, int r);
hipError_t launch_fp8_grad(const Fp8GradParams& p, hipStream_t stream);

}  // namespace qlora
