// Backward of the residual norm (norm.hip).  With n = h' r and m = block r_b:
//   dh  = dh' + r (weight dx - n mean(weight dx n))            the gradient of h' and of h
//   dp  = scale gate dh
//   dblock = dp, or with a norm behind the block
//          = r_b (post_weight dp - m mean(post_weight dp m))
//   dweight = sum_t dx n;  with C = sum_t dh m
//   dgate = scale post_weight C,  dpost_weight = scale gate C
// The two means come from sums that need no other mean, in one reduction: with
// c = scale gate post_weight,
//   sum c dh m = sum c m (dh' + r weight dx) - r mean(weight dx n) sum c m n
// A workgroup owns every G-th token and a thread the same eight (or twice
// eight) channels of all of them, so the sums over tokens stay in its registers
// until the end, and the next token's pieces load while this one's are summed;
// the workgroups' sums are then added in their order by a second kernel (no
// atomics).  dx, h', dh' and block are read once, dh and dblock written once.
// Bound by HBM: 4096 x 8192 bf16 (335 MB) in 57 us with the second kernel's 5, 5.9
// TB/s; with a norm behind the block and a gate (403 MB) 76; 1333 x 4096 in fp32
// with both (98 MB) 28, of it 5.6 the second.  Rows of 512 channels and fewer have
// one wave to a workgroup, 512 waves for 1024 SIMDs: 65536 x 512 bf16 105 us, 3.2
// TB/s; 32768 x 1024 72, 16384 x 2048 59.
#include <type_traits>

#include "norm.hpp"
#include "trace.hpp"
#include "wave.hpp"

namespace qlora {
namespace {

using namespace norm;

// What the call reads of a block: nothing of it where it has neither a norm nor
// a gate's gradient, whose dblock is a multiple of dh.
enum Block { kNoBlock, kPlainBlock, kGatedBlock, kNormedBlock };

template <int FS, int B, bool PAST>
struct Token {
  Eight<kWeightBf16> dx, block;
  Eight<FS> h, later;
  __device__ __forceinline__ void load(const NormParams& P, int64_t i, bool in) {
    if (!in) {
      dx.zero();
      h.zero();
      later.zero();
      block.zero();
      return;
    }
    dx.template load<PAST>(P.dx, i);
    h.template load<PAST>(P.h_out, i);
    if (P.dh_out) later.template load<PAST>(P.dh_out, i);
    else later.zero();
    if constexpr (B >= kGatedBlock) block.template load<PAST>(P.block, i);
  }
};

// weight and c = scale gate post_weight of a thread's eight channels
template <int FW, int B>
__device__ __forceinline__ void factors(const NormParams& P, int p, bool in, float (&w)[8], float (&c)[8]) {
  Eight<FW> t;
  t.zero();
  if (in) t.load(P.weight, 8 * p);
  t.values(w);
  if constexpr (B > kNoBlock) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = P.scale;
    float v[8];
    if (P.gate && in) {
      t.load(P.gate, 8 * p);
      t.values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] *= v[e];
    }
    if (B == kNormedBlock && in) {
      t.load(P.post_weight, 8 * p);
      t.values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] *= v[e];
    }
  }
}

// NP: pieces of eight channels a thread holds.  With one, its factors stay in
// registers and the next token's pieces are on their way; with two (more than
// 8192 channels) there is no room for either.  The bound of 1024 threads leaves
// 128 registers.  With a norm behind the block an fp32 stream spills two of them
// with one piece; two pieces spill 18 to 23, and three with a gate's gradient and
// all in fp32: 2048 x 16384 fp32, normed and gated (604 MB), takes 186 us, 3.2
// TB/s, without either (537 MB) 114.
template <int FS, int FW, int NP, int B, bool PAST>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormParams P) {
  __shared__ float4 slot[2][16];  // by token in turn: the one before may still be read
  const int pieces = P.D / 8, step = (int)blockDim.x, tid = (int)threadIdx.x, waves = step >> 6;
  float dw[NP][8], dc[NP][8];
#pragma unroll
  for (int u = 0; u < NP; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[u][e] = dc[u][e] = 0.0f;
  float w[8], c[8];
  if constexpr (NP == 1) factors<FW, B>(P, tid, tid < pieces, w, c);
  const float inv = 1.0f / (float)P.D;
  Token<FS, B, PAST> now[NP], next[NP];
  float2 r_now = {}, r_next = {};
  const auto load = [&](int64_t t, Token<FS, B, PAST>(&to)[NP], float2& r) {
#pragma unroll
    for (int u = 0; u < NP; ++u) to[u].load(P, t * P.D + 8 * (u * step + tid), u * step + tid < pieces);
    r = float2{P.stats[2 * t], P.stats[2 * t + 1]};
  };
  if constexpr (NP == 1) load(blockIdx.x, next, r_next);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x, turn ^= 1) {
    if constexpr (NP == 1) {
      now[0] = next[0];
      r_now = r_next;
      if (t + gridDim.x < P.T) load(t + gridDim.x, next, r_next);
    } else {
      load(t, now, r_now);
    }
    const float r = r_now.x, r_b = B == kNormedBlock ? r_now.y : 1.0f;
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      float dx[8], n[8], later[8], m[8];
      if constexpr (NP > 1) factors<FW, B>(P, u * step + tid, u * step + tid < pieces, w, c);
      now[u].dx.values(dx);
      now[u].h.values(n);
      if constexpr (B == kNormedBlock) {
        now[u].later.values(later);
        now[u].block.values(m);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= r;
        const float dn = dx[e] * w[e];
        s1 = __builtin_fmaf(dn, n[e], s1);
        if constexpr (B == kNormedBlock) {
          const float cm = c[e] * m[e];
          s2 = __builtin_fmaf(cm, __builtin_fmaf(r, dn, later[e]), s2);
          s3 = __builtin_fmaf(cm, n[e], s3);
        }
      }
    }
    s1 = wave::sum(s1);
    if constexpr (B == kNormedBlock) {
      s2 = wave::sum(s2);
      s3 = wave::sum(s3);
    }
    if (waves > 1) {
      if ((tid & 63) == 0) slot[turn][tid >> 6] = float4{s1, s2, s3, 0.0f};
      __syncthreads();
      s1 = s2 = s3 = 0.0f;
      for (int v = 0; v < waves; ++v) {
        const float4 x = slot[turn][v];
        s1 += x.x;
        s2 += x.y;
        s3 += x.z;
      }
    }
    const float mean = s1 * inv;
    // mean(c dh m) r_b, the factor of block in dblock / r_b: from the left, so that each r_b meets a block's size and no
    // power of it leaves the range
    const float mean_p = r_b * inv * __builtin_fmaf(-r * mean, s3, s2) * r_b;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = u * step + tid;
      const bool in = p < pieces;
      float dx[8], n[8], d[8];
      if constexpr (NP > 1) factors<FW, B>(P, p, in, w, c);
      now[u].dx.values(dx);
      now[u].h.values(n);
      now[u].later.values(d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= r;
        dw[u][e] = __builtin_fmaf(dx[e], n[e], dw[u][e]);
        d[e] = __builtin_fmaf(r, __builtin_fmaf(-mean, n[e], dx[e] * w[e]), d[e]);
      }
      if (in) store8<FS, PAST>(P.dh, t * P.D + 8 * p, d);
      if constexpr (B > kNoBlock) {
        float m[8];
        if constexpr (B >= kGatedBlock) {
          now[u].block.values(m);
#pragma unroll
          for (int e = 0; e < 8; ++e) dc[u][e] = __builtin_fmaf(d[e], m[e] * r_b, dc[u][e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] *= c[e];
          if constexpr (B == kNormedBlock) d[e] = r_b * __builtin_fmaf(-mean_p, m[e], d[e]);
        }
        if (in) store8<kWeightBf16>(P.dblock, t * P.D + 8 * p, d);
      }
    }
  }
  if (!P.dweight) return;
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int p = u * step + tid;
    if (p >= pieces) continue;
    store8<kWeightF32>(P.part, (2 * (int64_t)blockIdx.x) * P.D + 8 * p, dw[u]);
    if (B >= kGatedBlock) store8<kWeightF32>(P.part, (2 * (int64_t)blockIdx.x + 1) * P.D + 8 * p, dc[u]);
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

// Threads of a workgroup, and workgroups: two to a CU up to 2048 channels, one
// above, each with the same number of tokens or one less.  us of both kernels
// with one and two to a CU: 8192 x 2048 normed 45 42; 4096 x 4096 35 35; 1333 x
// 4096 (fp32, normed and gated) 25.5 26.9, 600 of them 17.8 19.9; 4096 x 8192 65
// 67; 8192 x 1024 (fp32, normed) with two and four 36 37.
int bwd_threads(int64_t D) { return (int)((D / 8 / (D > 8192 ? 2 : 1) + 63) / 64 * 64); }
int64_t bwd_groups(int64_t T, int64_t D) {
  const int64_t most = D <= 2048 ? 512 : 256, turns = (T + most - 1) / most;
  return turns ? (T + turns - 1) / turns : 0;
}

template <int N>
using Int = std::integral_constant<int, N>;

}  // namespace

size_t norm_bwd_part_bytes(int64_t T, int64_t D) { return (size_t)(bwd_groups(T, D) * 2 * D * (int64_t)sizeof(float)); }

hipError_t launch_norm_bwd(const NormParams& P, hipStream_t stream) {
  const int groups = (int)bwd_groups(P.T, P.D), threads = bwd_threads(P.D);
  // us of both kernels through and past the caches (all that is read, and dh; dblock is the next call's operand): 1024 x
  // 8192 bf16 19.1 20.4, 2048 of them 38.0 33.4, 4096 66.7 56.3, normed and gated 86.8 76.0; 1333 x 4096 fp32, normed
  // and gated, 26.8 30.1
  const int64_t wide = P.stream == kWeightF32 ? 4 : 2, reads_block = P.post_weight || P.dgate ? 2 : 0;
  const bool past = P.T * P.D * (2 + (P.dh_out ? 3 : 2) * wide + (P.block ? 2 : 0) + reads_block) >= kPastBytes;
  const auto go = [&](auto fs, auto fw, auto b) {
    constexpr int FS = decltype(fs)::value, FW = decltype(fw)::value, B = decltype(b)::value;
    const dim3 grid((unsigned)groups), block((unsigned)threads);
    if (P.D <= 8192) past ? launch(KID_NORM_BWD, k_norm_bwd<FS, FW, 1, B, true>, grid, block, stream, P)
                          : launch(KID_NORM_BWD, k_norm_bwd<FS, FW, 1, B, false>, grid, block, stream, P);
    else past ? launch(KID_NORM_BWD, k_norm_bwd<FS, FW, 2, B, true>, grid, block, stream, P)
              : launch(KID_NORM_BWD, k_norm_bwd<FS, FW, 2, B, false>, grid, block, stream, P);
    if (P.dweight) {
      const dim3 sums((unsigned)(P.D / 64), P.dgate || P.dpost_weight ? 2 : 1);
      launch(KID_NORM_SUM, k_norm_sum<FW>, sums, dim3(256), stream, P, groups);
    }
  };
  const auto by_formats = [&](auto b) {
    const Int<kWeightF32> f32;
    const Int<kWeightBf16> b16;
    if (P.stream == kWeightF32) P.weights == kWeightF32 ? go(f32, f32, b) : go(f32, b16, b);
    else P.weights == kWeightF32 ? go(b16, f32, b) : go(b16, b16, b);
  };
  if (!P.block) by_formats(Int<kNoBlock>());
  else if (P.post_weight) by_formats(Int<kNormedBlock>());
  else if (P.dgate) by_formats(Int<kGatedBlock>());
  else by_formats(Int<kPlainBlock>());
  return hipGetLastError();
}

}  // namespace qlora
