// The residual norm before and after a block; see norm.hip.
#pragma once

#include "common.hpp"

namespace qlora {

constexpr int64_t kNormMostCols = 16384;
constexpr int64_t kNormMostRows = ((int64_t)1 << 22) - 1;  // up to 1024 threads each, fewer than 2^32 in all

struct NormParams {
  int64_t T;
  int D;
  int stream;            // kWeightF32 or kWeightBf16: the format of h, h_out, dh, dh_out
  int weights;           // the same, of weight, post_weight and gate
  float eps, scale;
  const void* h;         // forward
  const uint16_t* block; // bf16 [T][D] or null
  const void* weight;
  const void* post_weight;  // null: no norm behind the block
  const void* gate;         // null: 1
  void* h_out;           // forward: written (null without a block); backward: read
  uint16_t* x;           // bf16 [T][D] or null
  uint8_t* codes;        // the 8-bit form by rows, or null
  uint8_t* scales;
  float* stats;          // [T][2]: 1 / rms of h_out, 1 / rms of block (1 without a norm behind it)
  // backward
  const uint16_t* dx;
  const void* dh_out;    // null: 0
  void* dh;
  uint16_t* dblock;      // null without a block
  float* dweight;        // fp32 [D], or null: no gradients of weight, post_weight and gate
  float* dpost_weight;
  float* dgate;
  int accumulate;
  float* part;           // norm_bwd_part_bytes
};

hipError_t launch_norm(const NormParams& p, hipStream_t stream);
size_t norm_bwd_part_bytes(int64_t T, int64_t D);
hipError_t launch_norm_bwd(const NormParams& p, hipStream_t stream);

namespace norm {

// A call that moves more than half of what the last-level cache holds (256 MB)
// takes the stream and the block past it: what is left of them there when they
// are read again is little, and takes the place of the next layer's input.
constexpr int64_t kPastBytes = (int64_t)128 << 20;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Eight consecutive elements: 16 bytes of bf16, 32 of fp32.
// PAST: not kept in the caches.
template <bool PAST>
__device__ __forceinline__ u32x4_t load16(const u32x4_t* q) {
  if constexpr (PAST) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool PAST>
__device__ __forceinline__ void store16(u32x4_t* q, u32x4_t v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, q);
  else *q = v;
}

template <int F>
struct Eight {
  u32x4_t a, b;
  template <bool PAST = false>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (F == kWeightF32) {
      const u32x4_t* q = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(p) + i);
      a = load16<PAST>(q);
      b = load16<PAST>(q + 1);
    } else {
      a = load16<PAST>(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i));
    }
  }
  __device__ __forceinline__ void zero() { a = b = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t x = a[q];
      if constexpr (F == kWeightF32) {
        const uint32_t y = b[q];
        f[q] = __builtin_bit_cast(float, x);
        f[4 + q] = __builtin_bit_cast(float, y);
      } else {
        f[2 * q] = __builtin_bit_cast(float, x << 16);
        f[2 * q + 1] = __builtin_bit_cast(float, x & 0xFFFF0000u);
      }
    }
  }
};

template <int F, bool PAST = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  if constexpr (F == kWeightF32) {
    u32x4_t* q = reinterpret_cast<u32x4_t*>(static_cast<float*>(p) + i);
    u32x4_t a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __builtin_bit_cast(uint32_t, f[e]);
      b[e] = __builtin_bit_cast(uint32_t, f[4 + e]);
    }
    store16<PAST>(q, a);
    store16<PAST>(q + 1, b);
  } else {
    store16<PAST>(
        reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i),
        u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])});
  }
}

}  // namespace norm
}  // namespace qlora
