// The gradient of the logits, for the layer's dY, from log probabilities of
// given tokens (weights d, and d_H of the entropy H) and from the distillation
// loss (weight g).  With log q = scale (z - M) - log S, both are
//   dz_j = scale * ( w_j - q_j (A_j + d_H (log q_j + H)) )
//   given tokens:  w_j = the d of entries that name j,  A = the sum of all d
//   distillation:  w_j = -g * (the p of entries that name j), and A = -g whole
//     for the listed tokens, -g (whole - ratio) for the others
// A row whose weights are all 0 has gradient 0, whatever its logits hold.
//
// The statistics of the row are known, so this is one pass: every logit is read
// once and every gradient written once, in pieces of 16 bytes.  A workgroup
// takes kGroupPieces pieces of one row.  Its entries with their logits are
// picked out before the first gradient is stored, so the gradients may take the
// logits' place; behind a barrier their gradients are written over the common
// ones, a thread to an entry.  Bound by HBM: 4096 x 128256 bf16 (1.05 GB read,
// 1.05 written) in 362 us, 5.8 TB/s, where a large copy reaches 5.0.
//
// A piece is read whole where the gradient's row starts as far from a 16-byte
// boundary as the logits' row does, and element by element otherwise: 4096 x
// 50257 bf16 of a head with 50304 columns take 129 us into rows of 50304, and
// 255 into rows of 50257.
#include <type_traits>

#include "logits.hpp"
#include "trace.hpp"
#include "wave.hpp"

namespace qlora {
namespace {

using namespace logits;

constexpr int kThreads = 256, kPieces = 4, kGroupPieces = kThreads * kPieces;

struct Shared {
  int64_t id[kLogitsMost];  // the group's entries: token, logit, weight
  float z[kLogitsMost], w[kLogitsMost];
  int count;
  float A, A_listed;
};

template <int F>
__device__ __forceinline__ u32x4_t pack(const float* f) {
  u32x4_t o;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (F == kWeightF32) {
      o[q] = __builtin_bit_cast(uint32_t, f[q]);
    } else if constexpr (F == kWeightBf16) {
      o[q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
    } else {
      const f16x2_t h = {(_Float16)f[2 * q], (_Float16)f[2 * q + 1]};
      o[q] = __builtin_bit_cast(uint32_t, h);
    }
  }
  return o;
}

template <int F>
__device__ __forceinline__ void store_element(char* row, int64_t i, float v) {
  if constexpr (F == kWeightF32) reinterpret_cast<float*>(row)[i] = v;
  else if constexpr (F == kWeightBf16) reinterpret_cast<uint16_t*>(row)[i] = f32_to_bf16_bits(v);
  else reinterpret_cast<_Float16*>(row)[i] = (_Float16)v;
}

// The weights of the row's entries, two to a lane of one wave, and A; the
// entries inside [i0, i1) go to LDS with their logits.
template <int F>
__device__ void entries(const LogitsGradParams& P, int64_t t, const Row<F>& row, int64_t i0, int64_t i1, Shared& sh) {
  const int lane = (int)threadIdx.x;
  int64_t id[2];
  bool in[2];
  float w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 64 * h;
    id[h] = i < P.n ? P.ids[t * P.n + i] : -1;
    in[h] = id[h] >= 0 && id[h] < P.in.vocab;
  }
  float A, A_listed;
  if (P.distill) {
    const float g = P.d_out[t], whole = P.stats[4 * t + 2], ratio = P.stats[4 * t + 3];
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) v[h] = in[h] ? P.values[t * P.n + lane + 64 * h] : kNone;
    float k = 1.0f;
    if (P.rest) {
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] = expf(v[h]);
    } else {
      const float most = fmaxf(wave::largest(fmaxf(v[0], v[1])), -kMost);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // v - most and what its rounding leaves (a far value's difference is off by its size times 2^-24)
        const float d = v[h] - most, back = d - v[h], left = (v[h] - (d - back)) - (most + back), x = expf(d);
        v[h] = x > 0.0f ? __builtin_fmaf(x, left, x) : 0.0f;
      }
      k = wave::sum(v[0] + v[1]);
      k = k > 0.0f ? 1.0f / k : 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = -g * (v[h] * k);
    A_listed = -g * whole;
    A = -g * (whole - ratio);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) w[h] = in[h] ? P.d_out[t * P.n + lane + 64 * h] : 0.0f;
    A = A_listed = wave::sum(w[0] + w[1]);
  }
  int n = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool mine = in[h] && id[h] >= i0 && id[h] < i1;
    const uint64_t who = __ballot(mine);
    if (mine) {
      const int at = n + __popcll(who & (((uint64_t)1 << lane) - 1));
      sh.id[at] = id[h];
      sh.w[at] = w[h];
      sh.z[at] = row.at(id[h]);
    }
    n += __popcll(who);
  }
  // no entries, or none with a weight (d_loss of a row without entries may be anything)
  const bool idle = __ballot(in[0] || in[1]) == 0 ||
                    (__ballot(w[0] != 0.0f || w[1] != 0.0f) == 0 && A == 0.0f && A_listed == 0.0f);
  if (lane == 0) {
    sh.count = idle ? -1 : n;
    sh.A = A;
    sh.A_listed = A_listed;
  }
}

template <int F, bool PAST>
__global__ __launch_bounds__(kThreads) void k_logits_grad(LogitsGradParams P, int groups) {
  constexpr int E = kPer<F>;
  __shared__ Shared sh;
  const int64_t t = (int64_t)blockIdx.x / groups;
  const int p0 = (int)(blockIdx.x - t * groups) * kGroupPieces;
  const Row<F> in(P.in.z, t, P.in.ld, (int)P.in.vocab), out(P.dz, t, P.out_ld, (int)P.out_cols);
  const int64_t first = (int64_t)p0 * E - out.head;
  if (threadIdx.x < 64) entries<F>(P, t, in, first, first + (int64_t)kGroupPieces * E, sh);
  __syncthreads();
  const float scale = P.in.scale;
  const int per = P.distill ? 4 : 2;
  const float M = P.stats[per * t], log_s = P.stats[per * t + 1];
  const float H = P.d_entropy ? P.entropy[t] : 0.0f, d_H = P.d_entropy ? P.d_entropy[t] : 0.0f;
  const bool none = M == kNone || (sh.count < 0 && d_H == 0.0f);
  const float A = sh.A, l2 = 1.44269504f;
  const auto gradient = [&](float z, float w, float a) {
    const float lq = __builtin_fmaf(z - M, scale, -log_s), q = __builtin_amdgcn_exp2f(lq * l2);
    float g = __builtin_fmaf(-q, a, w);
    // q first: where it is 0 the term is, however large d_H
    if (d_H != 0.0f) g = __builtin_fmaf(-d_H, q * (fmaxf(lq, -1e30f) + H), g);
    return scale * g;
  };
  char* const to = const_cast<char*>(out.start);
  const bool together = in.head == out.head;
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int p = p0 + u * kThreads + (int)threadIdx.x;
    if (p >= out.pieces) continue;
    const int64_t i0 = (int64_t)p * E - out.head;
    float f[E];
    if (none) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 0.0f;
    } else if (together && p >= in.full0 && p < in.full1) {
      unpack<F>(in.load(p), f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = gradient(f[e], 0.0f, A);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int64_t i = i0 + e;
        f[e] = i >= 0 && i < P.in.vocab ? gradient(in.at(i), 0.0f, A) : 0.0f;
      }
    }
    if (p >= out.full0 && p < out.full1) {
      u32x4_t* const dst = reinterpret_cast<u32x4_t*>(const_cast<char*>(out.aligned) + (int64_t)p * 16);
      if constexpr (PAST) __builtin_nontemporal_store(pack<F>(f), dst);
      else *dst = pack<F>(f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (i0 + e >= 0 && i0 + e < P.out_cols) store_element<F>(to, i0 + e, f[e]);
    }
  }
  if (none || sh.count <= 0) return;
  __syncthreads();
  const int mine = (int)threadIdx.x;
  if (mine >= sh.count) return;
  const int64_t id = sh.id[mine];
  float w = 0.0f;  // a token named twice has the weights of both, and both write the same
  for (int j = 0; j < sh.count; ++j) w += sh.id[j] == id ? sh.w[j] : 0.0f;
  store_element<F>(to, id, gradient(sh.z[mine], w, sh.A_listed));
}

}  // namespace

int64_t logits_grad_groups(int64_t T, int64_t out_cols, int format) {
  const int64_t per = format == kWeightF32 ? 4 : 8;
  const int64_t pieces = (out_cols + 2 * (per - 1)) / per;  // wherever the row starts
  return T * ((pieces + kGroupPieces - 1) / kGroupPieces);
}

hipError_t launch_logits_grad(const LogitsGradParams& P, hipStream_t stream) {
  if (P.in.T == 0) return hipSuccess;
  const int groups = (int)logits_grad_groups(1, P.out_cols, P.in.format);
  const dim3 grid((unsigned)(P.in.T * groups)), block(kThreads);
  // 4096 x 64000 bf16 (524 MB in, 524 out): 166 us past the caches, 175 through them; what reads 4096 x 128256
  // logits behind it takes 174 us, and 198.  217 x 50257 fp32 (44 MB each): 16.3 and 15.8.
  const bool past = 2 * P.in.T * P.in.bytes() >= kCacheBytes;  // logits and gradients
  const auto go = [&](auto f) {
    constexpr int F = decltype(f)::value;
    if (past) launch(KID_LOGITS_GRAD, k_logits_grad<F, true>, grid, block, stream, P, groups);
    else launch(KID_LOGITS_GRAD, k_logits_grad<F, false>, grid, block, stream, P, groups);
  };
  if (P.in.format == kWeightF32) go(std::integral_constant<int, kWeightF32>());
  else if (P.in.format == kWeightBf16) go(std::integral_constant<int, kWeightBf16>());
  else go(std::integral_constant<int, kWeightF16>());
  return hipGetLastError();
}

}  // namespace qlora
