// The residual norm: a block's output joins the residual stream, and the stream
// is normalised for the next layer's input.  Per token, over D channels:
//   m  = block * r_b,  r_b = 1 / sqrt(mean(block^2) + eps)    (m = block without a norm behind the block)
//   h' = h + scale * gate * post_weight * m
//   x  = (h' * r) * weight,  r = 1 / sqrt(mean(h'^2) + eps)
// x is formed from h' before h' is rounded to the stream's type, rounded once to
// bf16, or brought straight to the 8-bit form that the 8-bit layer reads (the
// same rule as k_fp8_quantize_rows, on x in fp32).
//
// A workgroup owns a token: every thread keeps its channels in registers
// through both sums, so h and block are read once and h' and x written once.
// Bound by HBM: 4096 x 8192 bf16 (268 MB) in 43 us, to the 8-bit form (235 MB)
// in 40, 5.9 TB/s; one token 2.4 us of a call's 11.
#include <type_traits>

#include "fp8_form.hpp"
#include "norm.hpp"
#include "trace.hpp"
#include "wave.hpp"

namespace qlora {
namespace {

using namespace norm;

__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  uint32_t o;
  o = __builtin_amdgcn_update_dpp(0, m, 0x128, 0xF, 0xF, false); m = o > m ? o : m;  // row_ror:8
  o = __builtin_amdgcn_update_dpp(0, m, 0x124, 0xF, 0xF, false); m = o > m ? o : m;
  o = __builtin_amdgcn_update_dpp(0, m, 0x122, 0xF, 0xF, false); m = o > m ? o : m;
  o = __builtin_amdgcn_update_dpp(0, m, 0x121, 0xF, 0xF, false); m = o > m ? o : m;
  return m;
}

// The sum over the workgroup, in every thread; slot: 16 floats that no other
// call of this launch uses.
__device__ __forceinline__ float block_sum(float v, float* slot) {
  v = wave::sum(v);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += slot[w];
  return s;
}

// NP: pieces of eight channels a thread holds
template <int FS, int FW, int NP, bool PAST>
__global__ __launch_bounds__(1024) void k_norm(NormParams P) {
  __shared__ float slot[2][16];
  const int64_t base = (int64_t)blockIdx.x * P.D;
  const int pieces = P.D / 8, step = (int)blockDim.x;
  float v[NP][8];
  float r_b = 1.0f;
  if (P.block) {
    float g[NP][8], ss = 0.0f;
    Eight<FS> h[NP];
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = u * step + (int)threadIdx.x;
      Eight<kWeightBf16> b;
      b.zero();
      h[u].zero();
      if (p < pieces) {
        b.template load<PAST>(P.block, base + 8 * p);
        h[u].template load<PAST>(P.h, base + 8 * p);
      }
      b.values(g[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(g[u][e], g[u][e], ss);
    }
    if (P.post_weight) r_b = rsqrtf(block_sum(ss, slot[0]) / (float)P.D + P.eps);
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = u * step + (int)threadIdx.x;
      float w[8];
      if (P.post_weight && p < pieces) {
        Eight<FW> t;
        t.load(P.post_weight, 8 * p);
        t.values(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[u][e] *= r_b * w[e];
      }
      if (P.gate && p < pieces) {
        Eight<FW> t;
        t.load(P.gate, 8 * p);
        t.values(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[u][e] *= w[e];
      }
      h[u].values(v[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] = __builtin_fmaf(P.scale, g[u][e], v[u][e]);
      if (p < pieces) store8<FS, PAST>(P.h_out, base + 8 * p, v[u]);
    }
  } else {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = u * step + (int)threadIdx.x;
      Eight<FS> h;
      h.zero();
      if (p < pieces) h.template load<PAST>(P.h, base + 8 * p);
      h.values(v[u]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int u = 0; u < NP; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[u][e], v[u][e], ss);
  const float r = rsqrtf(block_sum(ss, slot[1]) / (float)P.D + P.eps);
  if (threadIdx.x == 0) {
    P.stats[2 * (int64_t)blockIdx.x] = r;
    P.stats[2 * (int64_t)blockIdx.x + 1] = r_b;
  }
  const int64_t scale_ld = fp8_scale_ld(P.D);
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int p = u * step + (int)threadIdx.x;
    if (p < pieces) {
      Eight<FW> t;
      float w[8];
      t.load(P.weight, 8 * p);
      t.values(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] = v[u][e] * r * w[e];
      if (P.x) store8<kWeightBf16>(P.x, base + 8 * p, v[u]);
    }
    if (P.codes) {
      // 16 lanes to a block of 128 channels, a wave to four of them: one dword of scales
      const uint32_t e = fp8::scale_byte(row16_max(p < pieces ? fp8::absmax8(v[u]) : 0u));
      if (p < pieces) *reinterpret_cast<fp8::u32x2_t*>(P.codes + base + 8 * p) = fp8::codes8(v[u], e);
      const uint32_t b = p < pieces ? e : 127u;  // a block past the row's end
      const uint32_t word = (uint32_t)__builtin_amdgcn_readlane((int)b, 0) |
                            ((uint32_t)__builtin_amdgcn_readlane((int)b, 16) << 8) |
                            ((uint32_t)__builtin_amdgcn_readlane((int)b, 32) << 16) |
                            ((uint32_t)__builtin_amdgcn_readlane((int)b, 48) << 24);
      if ((threadIdx.x & 63) == 0 && p < pieces)
        reinterpret_cast<uint32_t*>(P.scales)[(int64_t)blockIdx.x * (scale_ld / 4) + p / 64] = word;
    }
  }
}

}  // namespace

hipError_t launch_norm(const NormParams& P, hipStream_t stream) {
  if (P.T == 0) return hipSuccess;
  const int pieces = P.D / 8;
  // Two pieces to a thread where there are more tokens than the CUs take at once; fewer tokens have more threads
  // each.  us with one and two: 4096 x 8192 bf16 44.3 42.5, to the 8-bit form 44.1 38.2, normed and gated 52.2 46.6;
  // 4096 x 5120 normed and gated 34.6 30.9; 1333 x 4096 fp32 18.2 17.8; 256 x 4096 fp32 7.8 9.0.  Four are as fast as
  // two or slower (42.8, 39.6, 48.2, 32.3, 18.8).
  const int np = pieces > 1024 || (P.T > 512 && pieces >= 128) ? 2 : 1;
  // tokens of 8192 bf16 channels, us through and past the caches: 1024 11.4 13.7, 2048 23.9 24.3, 2560 32.7 28.8, 4096
  // 48.7 43.1 (to the 8-bit form 44.6 39.7)
  const int64_t wide = P.stream == kWeightF32 ? 4 : 2;
  const bool past = P.T * P.D * ((P.block ? 2 * wide + 2 : wide) + (P.x ? 2 : 0) + (P.codes ? 1 : 0)) >= kPastBytes;
  const int threads = ((pieces + np - 1) / np + 63) / 64 * 64;
  const dim3 grid((unsigned)P.T), block((unsigned)threads);
  const auto go = [&](auto fs, auto fw) {
    constexpr int FS = decltype(fs)::value, FW = decltype(fw)::value;
    if (np == 1) past ? launch(KID_NORM, k_norm<FS, FW, 1, true>, grid, block, stream, P)
                      : launch(KID_NORM, k_norm<FS, FW, 1, false>, grid, block, stream, P);
    else past ? launch(KID_NORM, k_norm<FS, FW, 2, true>, grid, block, stream, P)
              : launch(KID_NORM, k_norm<FS, FW, 2, false>, grid, block, stream, P);
  };
  const std::integral_constant<int, kWeightF32> f32;
  const std::integral_constant<int, kWeightBf16> b16;
  if (P.stream == kWeightF32) P.weights == kWeightF32 ? go(f32, f32) : go(f32, b16);
  else P.weights == kWeightF32 ? go(b16, f32) : go(b16, b16);
  return hipGetLastError();
}

}  // namespace qlora
