// Backward of the residual norm (norm.hip).  With n = h' r and m = block r_b:
//   dh  = dh' + r (weight dx - n mean(weight dx n))            the gradient of h' and of h
//   dp  = scale gate dh
//   dblock = dp, or with a norm behind the block
//          = r_b (post_weight dp - m mean(post_weight dp m))
//   dweight = sum_t dx n;  with C = sum_t dh m
//   dgate = scale post_weight C,  dpost_weight = scale gate C
// A workgroup owns every G-th token and a thread the same eight (or twice
// eight) channels of all of them, so the sums over tokens stay in its registers
// until the end; the workgroups' sums are then added in their order by a second
// kernel (no atomics).  dx, h', dh' and block are read once, dh and dblock
// written once.
#include <type_traits>

#include "norm.hpp"
#include "trace.hpp"
#include "wave.hpp"

namespace qlora {
namespace {

using namespace norm;

constexpr int kGroups = 256;

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

template <int F>
__device__ __forceinline__ void values_at(const void* p, int64_t i, bool in, float (&f)[8]) {
  Eight<F> v;
  v.zero();
  if (in) v.load(p, i);
  v.values(f);
}

// BLOCK: 0 none, 1 a block, 2 a block with a norm behind it
template <int FS, int FW, int NP, int BLOCK>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormParams P) {
  __shared__ float slot[2][2][16];  // by token in turn: the one before may still be read
  const int pieces = P.D / 8, step = (int)blockDim.x;
  float dw[NP][8], dc[NP][8];
#pragma unroll
  for (int u = 0; u < NP; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[u][e] = dc[u][e] = 0.0f;
  const float inv = 1.0f / (float)P.D;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x, turn ^= 1) {
    const int64_t base = t * P.D;
    const float r = P.stats[2 * t], r_b = BLOCK == 2 ? P.stats[2 * t + 1] : 1.0f;
    float dn[NP][8], n[NP][8], s = 0.0f;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = u * step + (int)threadIdx.x;
      const bool in = p < pieces;
      float dx[8], w[8];
      values_at<kWeightBf16>(P.dx, base + 8 * p, in, dx);
      values_at<FS>(P.h_out, base + 8 * p, in, n[u]);
      values_at<FW>(P.weight, 8 * p, in, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[u][e] *= r;
        dw[u][e] = __builtin_fmaf(dx[e], n[u][e], dw[u][e]);
        dn[u][e] = dx[e] * w[e];
        s = __builtin_fmaf(dn[u][e], n[u][e], s);
      }
    }
    const float mean = block_sum(s, slot[turn][0]) * inv;
    float sp = 0.0f;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = u * step + (int)threadIdx.x;
      const bool in = p < pieces;
      float d[8];
      if (P.dh_out) {
        values_at<FS>(P.dh_out, base + 8 * p, in, d);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = __builtin_fmaf(r, __builtin_fmaf(-mean, n[u][e], dn[u][e]), d[e]);
      if (in) store8<FS>(P.dh, base + 8 * p, d);
      if constexpr (BLOCK > 0) {
        float g[8], w[8];
        if (P.gate) {
          values_at<FW>(P.gate, 8 * p, in, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] *= P.scale;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = P.scale;
        }
        if (BLOCK == 2 || (P.dgate && P.dweight)) {
          // n holds m, dn the gradient of m from here on
          values_at<kWeightBf16>(P.block, base + 8 * p, in, n[u]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            n[u][e] *= r_b;
            dc[u][e] = __builtin_fmaf(d[e], n[u][e], dc[u][e]);
          }
        }
        if constexpr (BLOCK == 2) values_at<FW>(P.post_weight, 8 * p, in, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dn[u][e] = d[e] * g[e];
          if constexpr (BLOCK == 2) {
            dn[u][e] *= w[e];
            sp = __builtin_fmaf(dn[u][e], n[u][e], sp);
          }
        }
        if constexpr (BLOCK == 1)
          if (in) store8<kWeightBf16>(P.dblock, base + 8 * p, dn[u]);
      }
    }
    if constexpr (BLOCK == 2) {
      const float mean_p = block_sum(sp, slot[turn][1]) * inv;
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const int p = u * step + (int)threadIdx.x;
#pragma unroll
        for (int e = 0; e < 8; ++e) dn[u][e] = r_b * __builtin_fmaf(-mean_p, n[u][e], dn[u][e]);
        if (p < pieces) store8<kWeightBf16>(P.dblock, base + 8 * p, dn[u]);
      }
    }
  }
  if (!P.dweight) return;
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int p = u * step + (int)threadIdx.x;
    if (p >= pieces) continue;
    store8<kWeightF32>(P.part, (2 * (int64_t)blockIdx.x) * P.D + 8 * p, dw[u]);
    if (BLOCK > 0) store8<kWeightF32>(P.part, (2 * (int64_t)blockIdx.x + 1) * P.D + 8 * p, dc[u]);
  }
}

// The workgroups' sums in their order: 16 threads along 64 channels, 16 ranges
// of the workgroups.
template <int FW>
__global__ __launch_bounds__(256) void k_norm_sum(NormParams P, int groups) {
  __shared__ float4 sums[16][16];
  const int x = (int)threadIdx.x & 15, y = (int)threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 64 + 4 * x;
  const int which = (int)blockIdx.y;
  float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  const int each = (groups + 15) / 16, g1 = (y + 1) * each < groups ? (y + 1) * each : groups;
#pragma unroll 8
  for (int g = y * each; g < g1; ++g) {
    const float4 v = *reinterpret_cast<const float4*>(P.part + (2 * (int64_t)g + which) * P.D + col);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  sums[y][x] = s;
  __syncthreads();
  if (y != 0) return;
  for (int q = 1; q < 16; ++q) {
    const float4 v = sums[q][x];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
  const auto weight = [&](const void* p, int e) {
    if (!p) return 1.0f;
    if constexpr (FW == kWeightF32) return static_cast<const float*>(p)[col + e];
    return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[col + e]);
  };
  const auto put = [&](float* to, int e, float d) { to[col + e] = P.accumulate ? to[col + e] + d : d; };
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (which == 0) {
      put(P.dweight, e, v[e]);
    } else {
      const float c = P.scale * v[e];
      if (P.dgate) put(P.dgate, e, c * weight(P.post_weight, e));
      if (P.dpost_weight) put(P.dpost_weight, e, c * weight(P.gate, e));
    }
  }
}

}  // namespace

size_t norm_bwd_part_bytes(int64_t T, int64_t D) {
  return (size_t)((T < kGroups ? T : kGroups) * 2 * D * (int64_t)sizeof(float));
}

hipError_t launch_norm_bwd(const NormParams& P, hipStream_t stream) {
  const int pieces = P.D / 8;
  const int np = pieces > 1024 ? 2 : 1;
  const int threads = ((pieces + np - 1) / np + 63) / 64 * 64;
  const int groups = (int)(P.T < kGroups ? P.T : kGroups);
  const int mode = !P.block ? 0 : P.post_weight ? 2 : 1;
  const auto go = [&](auto fs, auto fw, auto b) {
    constexpr int FS = decltype(fs)::value, FW = decltype(fw)::value, B = decltype(b)::value;
    const dim3 grid((unsigned)groups), block((unsigned)threads);
    if (np == 1) launch(KID_NORM_BWD, k_norm_bwd<FS, FW, 1, B>, grid, block, stream, P);
    else launch(KID_NORM_BWD, k_norm_bwd<FS, FW, 2, B>, grid, block, stream, P);
    if (P.dweight) {
      const dim3 sums((unsigned)(P.D / 64), P.dgate || P.dpost_weight ? 2 : 1);
      launch(KID_NORM_SUM, k_norm_sum<FW>, sums, dim3(256), stream, P, groups);
    }
  };
  const std::integral_constant<int, kWeightF32> f32;
  const std::integral_constant<int, kWeightBf16> b16;
  const auto by_weights = [&](auto b) {
    if (P.stream == kWeightF32) P.weights == kWeightF32 ? go(f32, f32, b) : go(f32, b16, b);
    else P.weights == kWeightF32 ? go(b16, f32, b) : go(b16, b16, b);
  };
  if (mode == 0) by_weights(std::integral_constant<int, 0>());
  else if (mode == 1) by_weights(std::integral_constant<int, 1>());
  else by_weights(std::integral_constant<int, 2>());
  return hipGetLastError();
}

}  // namespace qlora
