// Products of two 8-bit forms (fp8.hip): the base product of a linear layer on
// an 8-bit weight and its input gradient, with the adapter's rank-r term as a
// tail of the same fp32 accumulators:
//   C[t][n] = bf16( sum_k X[t][k] W[n][k] + sum_c At[t][c] Bt[n][c] )
//   C[t][k] = bf16( sum_n X[t][n] W[n][k] + sum_c At[t][c] Bt[k][c] )   (dx)
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 codes and
// both operands' scales: one instruction is one block of 128, and since a
// block's scale is the same for all its 128 elements, the order in which they
// are spread over the lanes is free as long as both operands use the same one.
// Lane l holds 32 codes of row (column) l % 16 and its scale byte; here lane
// group g = l / 16 takes the 16-byte chunks g and g + 4 of the 128.  The first
// operand is the weight, so a lane's four results are four consecutive output
// features of one token.
//
// Precision: the unit adds products in groups of eight aligned to the group's
// largest, dropping what lies below 2^-13 of it (measured), and everything
// after that in fp32.  A dropped bit is at most 2^-13 of one product, against
// the 2^-4 that each code is already rounded by and the 2^-8 of the result.
#include "dma.hpp"
#include "fp8.hpp"
#include "fp8_tail.hpp"
#include "trace.hpp"

namespace qlora {
namespace {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef int v2i_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v2i_t lds_v2i_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;
using dma::copy16;
using dma::kOob;
using dma::rsrc;
using dma::v4i_t;
using dma::wait_vm;

__device__ __forceinline__ f32x4_t mfma8(v8i_t a, v8i_t b, f32x4_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ v8i_t join(u32x4_t a, u32x4_t b) {
  return v8i_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

struct Fp8Launch {
  Fp8Params p;
  int32_t mt, nt;      // feature tiles, token tiles
  int32_t nsplit;      // contraction ranges
  int32_t steps, steps_per_split;
  int64_t out_cols;    // features: Nw, or Kw for dx
};

// ---------------------------------------------------------------------------
// 128 features x 128 tokens, four waves of 64 x 64, contraction steps of 128
// double-buffered in LDS.
// ---------------------------------------------------------------------------
constexpr int BT = 128;
constexpr int kTileBytes = BT * 128;
constexpr int kOutLd = BT + 8;

__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

template <bool DX>
__global__ __launch_bounds__(256) void k_fp8_tile(Fp8Launch L) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * kTileBytes];
  const Fp8Params& p = L.p;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int i = lane & 15, g = lane >> 4;
  const int wf = (wave & 1) * 64, wt = (wave >> 1) * 64;  // the wave's features and tokens
  int b = (int)blockIdx.x;
  const int split = b / (L.mt * L.nt);
  b -= split * (L.mt * L.nt);
  const int64_t f0 = (int64_t)(b % L.mt) * BT, t0 = (int64_t)(b / L.mt) * BT;
  const int64_t len = DX ? p.Nw : p.Kw;       // contraction
  const int64_t feats = DX ? p.Kw : p.Nw;
  const int s_begin = split * L.steps_per_split;
  const int s_end = s_begin + L.steps_per_split < L.steps ? s_begin + L.steps_per_split : L.steps;

  const v4i_t rx = rsrc(p.X + t0 * len, (p.T - t0) * len);
  const v4i_t rw = DX ? rsrc(p.W + f0, p.Nw * p.Kw - f0) : rsrc(p.W + f0 * p.Kw, (p.Nw - f0) * p.Kw);
  const uint32_t lds0 = LDS_ADDR(lds);

  auto issue = [&](int s) {
    const uint32_t st = lds0 + (uint32_t)((s & 1) * 2 * kTileBytes);
    const int64_t k0 = (int64_t)s * 128;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int blk = 4 * wave + q;
      const int R = 8 * blk + (lane >> 3);
      const int px = (lane & 7) ^ swz(R);
      const uint32_t vx = k0 + px * 16 < len && t0 + R < p.T ? (uint32_t)(R * len + k0 + px * 16) : kOob;
      copy16(rx, vx, st + kTileBytes + blk * 1024);
      uint32_t vw;
      if (DX) {
        const int pw = (lane & 7) ^ (R & 7);
        vw = k0 + R < p.Nw && f0 + pw * 16 < p.Kw ? (uint32_t)((k0 + R) * p.Kw + pw * 16) : kOob;
      } else {
        vw = k0 + px * 16 < len && f0 + R < p.Nw ? (uint32_t)(R * p.Kw + k0 + px * 16) : kOob;
      }
      copy16(rw, vw, st + blk * 1024);
    }
  };

  f32x4_t acc[4][4];  // [feature tile][token tile]
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[a][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int64_t ldx = fp8_scale_ld(len), ldw = fp8_scale_ld(p.Kw);
  if (s_begin < s_end) issue(s_begin);
  for (int s = s_begin; s < s_end; ++s) {
    wait_vm<0>();
    __syncthreads();
    uint32_t sx[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t t = t0 + wt + 16 * c + i;
      sx[c] = p.Xs[(t < p.T ? t : p.T - 1) * ldx + s];
    }
    const uint32_t sw = DX ? p.Ws[(int64_t)s * ldw + (f0 >> 7)] : p.Ws[(f0 >> 7) * ldw + s];
    if (s + 1 < s_end) issue(s + 1);
    const uint8_t* w = lds + (s & 1) * 2 * kTileBytes;
    const uint8_t* x = w + kTileBytes;
    v8i_t fx[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int R = wt + 16 * c + i;
      fx[c] = join(*reinterpret_cast<const u32x4_t*>(x + R * 128 + ((g ^ swz(R)) << 4)),
                   *reinterpret_cast<const u32x4_t*>(x + R * 128 + (((g + 4) ^ swz(R)) << 4)));
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      v8i_t fw;
      if (DX) {
        // transposed: column wf + 16a + l%16, rows of chunks g and g + 4; 16
        // lanes read 8 rows of 16 bytes, lane i receives its column's 8 rows
        const int piece = (wf >> 4) + a;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int R = (q >> 1) * 64 + 16 * g + 8 * (q & 1) + (i >> 1);
          const v2i_t v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_v2i_t*)((lds_u8_t*)w + R * 128 + ((piece ^ (R & 7)) << 4) + 8 * (i & 1)));
          fw[2 * q] = v[0];
          fw[2 * q + 1] = v[1];
        }
      } else {
        const int R = wf + 16 * a + i;
        fw = join(*reinterpret_cast<const u32x4_t*>(w + R * 128 + ((g ^ swz(R)) << 4)),
                  *reinterpret_cast<const u32x4_t*>(w + R * 128 + (((g + 4) ^ swz(R)) << 4)));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][c] = mfma8(fw, fx[c], acc[a][c], sw, sx[c]);
    }
  }

  if (p.r > 0 && split == 0) {
    for (int c0 = 0; c0 < 2 * p.r; c0 += 32) {
      bf16x8_t bt[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) bt[c] = tail_token(p, t0 + wt + 16 * c + i, c0 + 8 * g);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const bf16x8_t wa = tail_weight(p, f0 + wf + 16 * a + i, feats, c0 + 8 * g);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa, bt[c], acc[a][c], 0, 0, 0);
      }
    }
  }

  if (L.nsplit > 1) {
    float* part = p.part + (int64_t)split * p.T * feats;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t t = t0 + wt + 16 * c + i, f = f0 + wf + 16 * a + 4 * g;
        if (t < p.T && f < feats) *reinterpret_cast<f32x4_t*>(part + t * feats + f) = acc[a][c];
      }
    return;
  }
  __syncthreads();
  uint16_t* out = reinterpret_cast<uint16_t*>(lds);  // [token][feature]
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f32x4_t v = acc[a][c];
      *reinterpret_cast<uint2*>(out + (wt + 16 * c + i) * kOutLd + wf + 16 * a + 4 * g) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  __syncthreads();
  for (int e = threadIdx.x; e < BT * BT / 8; e += 256) {
    const int R = e >> 4, col = (e & 15) * 8;
    if (t0 + R < p.T && f0 + col < feats)
      *reinterpret_cast<u32x4_t*>(p.C + (t0 + R) * feats + f0 + col) =
          *reinterpret_cast<const u32x4_t*>(out + R * kOutLd + col);
  }
}
static_assert(BT * kOutLd * 2 <= 4 * kTileBytes, "the output tile fits over the stages");

// The contraction ranges' partial sums in range order, rounded once; four
// consecutive elements a thread.
__global__ __launch_bounds__(256) void k_fp8_sum(const float* __restrict__ part, int nsplit, int64_t n,
                                                 uint16_t* __restrict__ C) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= n) return;
  float4 v = *reinterpret_cast<const float4*>(part + e);
  for (int q = 1; q < nsplit; ++q) {
    const float4 w = *reinterpret_cast<const float4*>(part + q * n + e);
    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
  }
  *reinterpret_cast<uint2*>(C + e) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__global__ __launch_bounds__(256) void k_fp8_pair(const uint16_t* __restrict__ M, int64_t rows, int r, int64_t ldh,
                                                  int transposed, uint16_t* __restrict__ out) {
  // 64 rows a workgroup; A's transpose goes through LDS so that both sides are
  // read and written along their rows
  __shared__ uint16_t t[64][130];
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int n = (int)(rows - r0 < 64 ? rows - r0 : 64);
  for (int e = threadIdx.x; e < 64 * r; e += 256) {
    if (transposed) {
      const int j = e >> 6, m = e & 63;
      if (m < n) t[m][j] = M[(int64_t)j * rows + r0 + m];
    } else {
      const int m = e / r, j = e - m * r;
      if (m < n) t[m][j] = M[(r0 + m) * r + j];
    }
  }
  __syncthreads();
  const int l = (int)ldh;
  for (int e = threadIdx.x; e < n * l; e += 256) {
    const int m = e / l, c = e - m * l;
    out[(r0 + m) * ldh + c] = c < r ? t[m][c] : (c < 2 * r ? t[m][c - r] : (uint16_t)0);
  }
}

// contraction ranges: as many workgroups as fill the 256 CUs twice, each range at least four steps
int product_splits(int64_t T, int64_t feats, int64_t len) {
  const int64_t tiles = ((T + BT - 1) / BT) * ((feats + BT - 1) / BT);
  const int64_t steps = (len + 127) / 128;
  int64_t s = 512 / tiles;
  if (s > steps / 4) s = steps / 4;
  if (s > 16) s = 16;
  return (int)(s < 1 ? 1 : s);
}

}  // namespace

size_t fp8_product_part_bytes(int64_t T, int64_t Nw, int64_t Kw, int dx) {
  const int64_t feats = dx ? Kw : Nw;
  const int s = product_splits(T, feats, dx ? Nw : Kw);
  return s > 1 ? (size_t)s * T * feats * 4 : 0;
}

hipError_t launch_fp8_product(const Fp8Params& p, hipStream_t stream) {
  if (((p.T + 255) / 256) * (((p.dx ? p.Kw : p.Nw) + 255) / 256) >= 128) return launch_fp8_wide(p, stream);
  Fp8Launch L{};
  L.p = p;
  const int64_t feats = p.dx ? p.Kw : p.Nw, len = p.dx ? p.Nw : p.Kw;
  L.out_cols = feats;
  L.mt = (int32_t)((feats + BT - 1) / BT);
  L.nt = (int32_t)((p.T + BT - 1) / BT);
  L.steps = (int32_t)((len + 127) / 128);
  L.nsplit = product_splits(p.T, feats, len);
  L.steps_per_split = (L.steps + L.nsplit - 1) / L.nsplit;
  if (L.nsplit > 1 && (!p.part || p.part_bytes < fp8_product_part_bytes(p.T, p.Nw, p.Kw, p.dx)))
    return hipErrorInvalidValue;
  {
    KernelEvents ev(KID_FP8_GEMM);
    const hipEvent_t e0 = ev.start(), e1 = ev.stop();
    const dim3 grid((unsigned)(L.mt * L.nt * L.nsplit));
    if (p.dx) hipExtLaunchKernelGGL(k_fp8_tile<true>, grid, dim3(256), 0, stream, e0, e1, 0, L);
    else hipExtLaunchKernelGGL(k_fp8_tile<false>, grid, dim3(256), 0, stream, e0, e1, 0, L);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || L.nsplit == 1) return e;
  const int64_t n = p.T * feats;
  KernelEvents ev(KID_REDUCE);
  hipExtLaunchKernelGGL(k_fp8_sum, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, ev.start(), ev.stop(),
                        0, p.part, L.nsplit, n, p.C);
  return hipGetLastError();
}

hipError_t launch_fp8_pair(const uint16_t* M, int64_t rows, int r, int64_t ldh, int transposed, uint16_t* out,
                           hipStream_t stream) {
  KernelEvents ev(KID_FP8_DOWN);
  hipExtLaunchKernelGGL(k_fp8_pair, dim3((unsigned)((rows + 63) / 64)), dim3(256), 0, stream, ev.start(), ev.stop(), 0,
                        M, rows, r, ldh, transposed, out);
  return hipGetLastError();
}

}  // namespace qlora
