// The operators on the logits of the last layer: parameters, and the reading
// of a row that they share.  See logits.hip (statistics, log probabilities,
// the distillation loss), logits_top.hpp (the largest of a row) and
// logits_grad.hip (gradients).
#pragma once

#include "common.hpp"

namespace qlora {

// The most tokens given per row, teacher's entries per row, and alternatives.
constexpr int kLogitsMost = 128;

struct LogitsRows {
  const void* z;   // rows of `vocab` logits, ld elements apart
  int format;      // kWeight*
  int64_t T, vocab, ld;
  float scale;     // q = softmax(scale * z)
  int64_t bytes() const { return vocab * (format == kWeightF32 ? 4 : 2); }  // of a row
};

// The last-level cache of the card.  Logits that it does not hold gain nothing
// from passing through it, and push out what others left there.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;

struct ScoreParams {
  LogitsRows in;
  int n;                  // tokens given per row
  const int64_t* tokens;  // [T][n]
  float* logprob;         // [T][n]
  float* stats;           // [T][2]
  float* entropy;         // [T] or null
  int top;
  int64_t* top_ids;       // [T][top]
  float* top_logprob;     // [T][top]
};
hipError_t launch_score(const ScoreParams& p, hipStream_t stream);

struct DistillParams {
  LogitsRows in;
  int k;
  const int64_t* ids;   // [T][k]
  const float* values;  // [T][k]
  int rest;
  float* loss;          // [T]
  float* stats;         // [T][4]
};
hipError_t launch_distill(const DistillParams& p, hipStream_t stream);

// The gradient of either: n given tokens with their weights, or the teacher's k entries.
struct LogitsGradParams {
  LogitsRows in;
  int n;
  const int64_t* ids;      // [T][n]
  const float* values;     // distillation: [T][n]
  int distill, rest;
  const float* stats;      // [T][2], distillation [T][4]
  const float* d_out;      // d_logprob [T][n], distillation d_loss [T]
  const float* entropy;    // [T] with d_entropy
  const float* d_entropy;  // [T] or null
  void* dz;                // rows of out_cols elements of the same format, out_ld apart
  int64_t out_cols, out_ld;
};
hipError_t launch_logits_grad(const LogitsGradParams& p, hipStream_t stream);
// Workgroups of the gradient's launch; at most kGradMostGroups.
int64_t logits_grad_groups(int64_t T, int64_t out_cols, int format);
constexpr int64_t kGradMostGroups = ((int64_t)1 << 24) - 1;  // 256 threads each, fewer than 2^32 in all
constexpr int64_t kLogitsMostRows = ((int64_t)1 << 22) - 1;  // up to 1024 threads each

namespace logits {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float kMost = 3.402823466e38f;  // the largest finite float
constexpr float kNone = -__builtin_inff();

template <int F>
constexpr int kPer = F == kWeightF32 ? 4 : 8;  // elements in a piece of 16 bytes
template <int F>
constexpr int kBytes = 16 / kPer<F>;

// The elements of one piece as fp32 (exact).
template <int F>
__device__ __forceinline__ void unpack(u32x4_t w, float* f) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t x = w[q];
    if constexpr (F == kWeightF32) {
      f[q] = __builtin_bit_cast(float, x);
    } else if constexpr (F == kWeightBf16) {
      f[2 * q] = __builtin_bit_cast(float, x << 16);
      f[2 * q + 1] = __builtin_bit_cast(float, x & 0xFFFF0000u);
    } else {
      const f16x2_t h = __builtin_bit_cast(f16x2_t, x);
      f[2 * q] = (float)h[0];
      f[2 * q + 1] = (float)h[1];
    }
  }
}

template <int F>
__device__ __forceinline__ float element(const char* row, int64_t i) {
  if constexpr (F == kWeightF32) return reinterpret_cast<const float*>(row)[i];
  const uint32_t h = reinterpret_cast<const uint16_t*>(row)[i];
  if constexpr (F == kWeightBf16) return bf16_bits_to_f32(h);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// A row as pieces of 16 bytes on 16-byte boundaries: piece p holds the elements
// p * kPer - head .. + kPer - 1.  Only the first and the last piece may reach
// past the row, and their elements are read one by one.
template <int F>
struct Row {
  const char* start;    // element 0
  const char* aligned;  // piece 0
  int head;             // elements of piece 0 before the row
  int vocab;
  int pieces, full0, full1;  // all pieces; the full ones full0 .. full1 - 1
  __device__ __forceinline__ Row(const void* z, int64_t row, int64_t ld, int vocab_) : vocab(vocab_) {
    start = static_cast<const char*>(z) + row * ld * kBytes<F>;
    const int off = (int)(reinterpret_cast<uintptr_t>(start) & 15);
    aligned = start - off;
    head = off / kBytes<F>;
    const int64_t end = (int64_t)vocab + head;
    pieces = (int)((end + kPer<F> - 1) / kPer<F>);
    full0 = head ? 1 : 0;
    full1 = (int)(end / kPer<F>);
    if (full1 < full0) full1 = full0;
  }
  template <bool PAST = false>  // not kept in the caches
  __device__ __forceinline__ u32x4_t load(int p) const {
    const u32x4_t* const q = reinterpret_cast<const u32x4_t*>(aligned + (int64_t)p * 16);
    if constexpr (PAST) return __builtin_nontemporal_load(q);
    return *q;
  }
  __device__ __forceinline__ float at(int64_t i) const { return element<F>(start, i); }
  // The elements outside the full pieces: [0, edge0) and [edge1, vocab), fewer than 2 * kPer.
  __device__ __forceinline__ int edge0() const { return full0 * kPer<F> - head < vocab ? (head ? kPer<F> - head : 0) : vocab; }
  __device__ __forceinline__ int edge1() const {
    const int64_t e = (int64_t)full1 * kPer<F> - head;
    return e < vocab ? (e > edge0() ? (int)e : edge0()) : vocab;
  }
  __device__ __forceinline__ int edges() const { return edge0() + vocab - edge1(); }
  __device__ __forceinline__ int edge(int q) const { return q < edge0() ? q : edge1() + q - edge0(); }
};

// Bits of a float in the order of the values, as an unsigned number; the two
// zeros alike, NaN below all else.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
  if (v != v) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  if (k == 0) return __builtin_nanf("");
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

}  // namespace logits
}  // namespace qlora
