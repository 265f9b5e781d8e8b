// The 8-bit form of a matrix M [R][C] and its kernels (gfx950).
//
// codes [R][C]: OCP e4m3 (largest 448, code 0x7F / 0xFF NaN).  One scale
// 2^(e - 127), stored as the byte e, for each block of 1 x 128 elements
// (activations, gradients) or 128 x 128 (weights); scales [R or ceil(R/128)]
// rows of 4 ceil(C/512) bytes, those past the last block holding 127.
//   m    = largest finite |x| of the block
//   e    = smallest byte in 1 .. 254 with m <= 448 * 2^(e - 127)
//   code = e4m3_rne(x * 2^(127 - e)); what is not finite becomes NaN
// m = 448 * 2^q has exponent q + 8 and mantissa 0x600000, so adding 0x1FFFFF
// to m's bits carries into the exponent field exactly when m's mantissa is
// above that: e = ((bits(m) + 0x1FFFFF) >> 23) - 8.
//
// The scales are powers of two because the matrix units of gfx950 multiply
// such scales in as they go (v_mfma_scale_*): a block of 128 then costs a
// product no vector instruction.  It costs no accuracy either: e4m3 is a
// floating format, so scaling by 2^q changes no relative rounding error; what
// is lost against a scale of m / 448 is at most one of 18 binades of range.
//
// All three kernels are bound by HBM: every element is read once and written
// once, with loads and stores of 8 or 16 bytes a lane.
#include "fp8.hpp"
#include "fp8_form.hpp"
#include "trace.hpp"

namespace qlora {
namespace {

using fp8::absmax8;
using fp8::codes8;
using fp8::scale_byte;
using fp8::u32x2_t;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// Eight consecutive elements as fp32 (exact).
template <int F>
struct Load8 {
  u32x4_t a, b;  // b: fp32 input only
  __device__ __forceinline__ void load(const void* M, int64_t elem) {
    if constexpr (F == kWeightF32) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(M) + elem);
      a = __builtin_nontemporal_load(p);
      b = __builtin_nontemporal_load(p + 1);
    } else {
      a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(M) + elem));
    }
  }
  __device__ __forceinline__ void zero() { a = b = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (F == kWeightF32) {
        const uint32_t lo = a[q], hi = b[q];
        f[q] = __builtin_bit_cast(float, lo);
        f[4 + q] = __builtin_bit_cast(float, hi);
      } else if constexpr (F == kWeightBf16) {
        f[2 * q] = __builtin_bit_cast(float, a[q] << 16);
        f[2 * q + 1] = __builtin_bit_cast(float, a[q] & 0xFFFF0000u);
      } else {
        const uint32_t w = a[q];
        const f16x2_t h = __builtin_bit_cast(f16x2_t, w);
        f[2 * q] = (float)h[0];
        f[2 * q + 1] = (float)h[1];
      }
    }
  }
};

// The largest of the 16 lanes of a row (DPP rotations).
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  uint32_t o;
  o = __builtin_amdgcn_update_dpp(0, m, 0x128, 0xF, 0xF, false); m = o > m ? o : m;  // row_ror:8
  o = __builtin_amdgcn_update_dpp(0, m, 0x124, 0xF, 0xF, false); m = o > m ? o : m;  // row_ror:4
  o = __builtin_amdgcn_update_dpp(0, m, 0x122, 0xF, 0xF, false); m = o > m ? o : m;  // row_ror:2
  o = __builtin_amdgcn_update_dpp(0, m, 0x121, 0xF, 0xF, false); m = o > m ? o : m;  // row_ror:1
  return m;
}

// 1 x 128 blocks.  A wave owns units of 512 columns of one row: 16 lanes to a
// block, 8 elements to a lane, the unit's four scales one dword.  So a row's
// unit is one load of 1 KB and one store of 512 bytes, and the largest value
// takes four rotations inside the 16 lanes.  4096 x 22016 bf16 (271 MB read and
// written): 44 us, 6.1 TB/s.
constexpr int kUnitsPerWave = 4;

template <int F>
__global__ __launch_bounds__(256) void k_fp8_quantize_rows(const void* __restrict__ M, int64_t cols,
                                                           uint32_t units_per_row, uint32_t units,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t u0 = (blockIdx.x * 4 + wave) * kUnitsPerWave;
  uint32_t row = u0 / units_per_row, cu = u0 - row * units_per_row;
  Load8<F> in[kUnitsPerWave];
  int64_t at[kUnitsPerWave];
  bool ok[kUnitsPerWave];
  // every load goes out before the first use; lanes past the row's or the
  // matrix's end read its first elements, which count as zero below
#pragma unroll
  for (int q = 0; q < kUnitsPerWave; ++q) {
    const int64_t col = (int64_t)cu * 512 + lane * 8;
    ok[q] = u0 + q < units && col < cols;
    at[q] = (int64_t)row * cols + col;
    in[q].load(M, ok[q] ? at[q] : 0);
    if (++cu == units_per_row) {
      cu = 0;
      ++row;
    }
  }
#pragma unroll
  for (int q = 0; q < kUnitsPerWave; ++q) {
    float f[8];
    in[q].values(f);
    const uint32_t m = row_max(ok[q] ? absmax8(f) : 0u);
    const uint32_t e = scale_byte(m);
    if (ok[q]) *reinterpret_cast<u32x2_t*>(codes + at[q]) = codes8(f, e);
    const uint32_t b = ok[q] ? e : 127u;  // a block past the row's end
    const uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)b, 0) | ((uint32_t)__builtin_amdgcn_readlane((int)b, 16) << 8) |
                       ((uint32_t)__builtin_amdgcn_readlane((int)b, 32) << 16) |
                       ((uint32_t)__builtin_amdgcn_readlane((int)b, 48) << 24);
    if (lane == 0 && u0 + q < units) reinterpret_cast<uint32_t*>(scales)[u0 + q] = w;
  }
}

// 128 x 128 blocks: a workgroup owns one, thread t the 8 columns 8 (t % 16) of
// rows t / 16, t / 16 + 16, ...; the block stays in registers (32 of them at 16
// bits) between the largest value and the codes, so it is read once.  22016 x
// 8192 bf16 (541 MB): 83 us repeated on one weight, 96 where weights take
// turns; 6.5 and 5.6 TB/s.
template <int F>
__global__ __launch_bounds__(256) void k_fp8_quantize_tiles(const void* __restrict__ M, int64_t rows, int64_t cols,
                                                            int32_t tiles_x, int64_t scale_ld,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ uint32_t wmax[4];
  const int ty = (int)blockIdx.x / tiles_x, tx = (int)blockIdx.x - ty * tiles_x;
  const int64_t row0 = (int64_t)ty * kFp8Block + (threadIdx.x >> 4);
  const int64_t col = (int64_t)tx * kFp8Block + (threadIdx.x & 15) * 8;
  Load8<F> in[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (col < cols && row0 + 16 * q < rows) in[q].load(M, (row0 + 16 * q) * cols + col);
    else in[q].zero();
  }
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float f[8];
    in[q].values(f);
    const uint32_t v = absmax8(f);
    m = v > m ? v : m;
  }
  m = row_max(m);
#pragma unroll
  for (int o = 16; o < 64; o *= 2) {
    const uint32_t v = __shfl_xor(m, o, 64);
    m = v > m ? v : m;
  }
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) m = wmax[w] > m ? wmax[w] : m;
  const uint32_t e = scale_byte(m);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float f[8];
    in[q].values(f);
    if (col < cols && row0 + 16 * q < rows)
      *reinterpret_cast<u32x2_t*>(codes + (row0 + 16 * q) * cols + col) = codes8(f, e);
  }
  // the last tile of a row of tiles also fills the row's padding
  const int last = tx == tiles_x - 1 ? (int)scale_ld : tx + 1;
  if (tx + (int)threadIdx.x < last) scales[ty * scale_ld + tx + threadIdx.x] = threadIdx.x == 0 ? (uint8_t)e : (uint8_t)127;
}

// Sixteen codes a thread.  4096 x 8192 (101 MB): 19 to 21 us, 5.0 TB/s, a
// copy's rate.
__global__ __launch_bounds__(256) void k_fp8_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, int64_t pieces,
                                                        int64_t pieces_per_row, int64_t scale_ld, int row_shift,
                                                        uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int64_t row = i / pieces_per_row;
  const int64_t piece = i - row * pieces_per_row;
  const u32x4_t c = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(codes) + i);
  const uint32_t e = scales[(row >> row_shift) * scale_ld + (piece >> 3)];
  const float k = __builtin_bit_cast(float, e << 23);
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o[2 * q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[q], k, false));
    o[2 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[q], k, true));
  }
  u32x4_t* dst = reinterpret_cast<u32x4_t*>(out) + 2 * i;
  dst[0] = u32x4_t{o[0], o[1], o[2], o[3]};
  dst[1] = u32x4_t{o[4], o[5], o[6], o[7]};
}

}  // namespace

hipError_t launch_fp8_quantize(const void* M, int format, int64_t rows, int64_t cols, int block_rows, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  KernelEvents ev(KID_FP8_QUANTIZE);
  const hipEvent_t e0 = ev.start(), e1 = ev.stop();
  if (block_rows == 1) {
    const int64_t upr64 = (cols + 511) / 512, units64 = rows * upr64;
    if (units64 >= (int64_t)1 << 27) return hipErrorInvalidValue;
    const uint32_t upr = (uint32_t)upr64, units = (uint32_t)units64;
    const dim3 grid((units + 4 * kUnitsPerWave - 1) / (4 * kUnitsPerWave));
    switch (format) {
      case kWeightF32: hipExtLaunchKernelGGL(k_fp8_quantize_rows<kWeightF32>, grid, dim3(256), 0, stream, e0, e1, 0, M, cols, upr, units, codes, scales); break;
      case kWeightBf16: hipExtLaunchKernelGGL(k_fp8_quantize_rows<kWeightBf16>, grid, dim3(256), 0, stream, e0, e1, 0, M, cols, upr, units, codes, scales); break;
      default: hipExtLaunchKernelGGL(k_fp8_quantize_rows<kWeightF16>, grid, dim3(256), 0, stream, e0, e1, 0, M, cols, upr, units, codes, scales); break;
    }
  } else {
    const int32_t tx = (int32_t)((cols + kFp8Block - 1) / kFp8Block);
    const int64_t ty = (rows + kFp8Block - 1) / kFp8Block, ld = fp8_scale_ld(cols);
    const dim3 grid((unsigned)(tx * ty));
    switch (format) {
      case kWeightF32: hipExtLaunchKernelGGL(k_fp8_quantize_tiles<kWeightF32>, grid, dim3(256), 0, stream, e0, e1, 0, M, rows, cols, tx, ld, codes, scales); break;
      case kWeightBf16: hipExtLaunchKernelGGL(k_fp8_quantize_tiles<kWeightBf16>, grid, dim3(256), 0, stream, e0, e1, 0, M, rows, cols, tx, ld, codes, scales); break;
      default: hipExtLaunchKernelGGL(k_fp8_quantize_tiles<kWeightF16>, grid, dim3(256), 0, stream, e0, e1, 0, M, rows, cols, tx, ld, codes, scales); break;
    }
  }
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                 int block_rows, uint16_t* out, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int64_t pieces = rows * cols / 16;
  KernelEvents ev(KID_FP8_DEQUANTIZE);
  hipExtLaunchKernelGGL(k_fp8_dequantize, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, stream, ev.start(),
                        ev.stop(), 0, codes, scales, pieces, cols / 16, fp8_scale_ld(cols), block_rows == 1 ? 0 : 7,
                        out);
  return hipGetLastError();
}

}  // namespace qlora
