// The largest elements of a row, ties to the lower index.
//
// An element's key is its value in the order of the floats (32 bits), then its
// index from the end (32 bits): no two are alike, so "the k largest" is one set
// in one order whatever the ties.
#pragma once

#include "logits.hpp"

namespace qlora {
namespace logits {

constexpr int kCandidates = 1024;

__device__ __forceinline__ uint64_t top_key(float v, int64_t i) {
  return ((uint64_t)ordered(v) << 32) | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ int64_t top_index(uint64_t key) { return (int64_t)(0xFFFFFFFFu - (uint32_t)key); }
__device__ __forceinline__ float top_value(uint64_t key) { return from_ordered((uint32_t)(key >> 32)); }

struct TopShared {
  uint64_t key[kCandidates];
  int count;
};

// Calls at(value, index) for the elements of pieces p0 .. p1 - 1 and, with
// `edges`, for those outside the full pieces.
template <int F, int THREADS, class At>
__device__ __forceinline__ void each_element(const Row<F>& row, int p0, int p1, bool edges, const At& at) {
  for (int p = p0 + (int)threadIdx.x; p < p1; p += THREADS) {
    float f[kPer<F>];
    unpack<F>(row.load(p), f);
    const int64_t i0 = (int64_t)p * kPer<F> - row.head;
#pragma unroll
    for (int e = 0; e < kPer<F>; ++e) at(f[e], i0 + e);
  }
  if (edges && (int)threadIdx.x < row.edges()) {
    const int i = row.edge((int)threadIdx.x);
    at(row.at(i), (int64_t)i);
  }
}

// Puts the elements of the pieces (and edges) with the K largest keys, and at
// most kCandidates in all, into sh.key; sh.count is their number.  Bisects on
// the key between `low` (at least K elements reach it) and `high` (none is
// above it): one pass over the pieces for each step.
template <int F, int THREADS>
__device__ void top_bisect(const Row<F>& row, int p0, int p1, bool edges, int K, uint64_t low, uint64_t high,
                           TopShared& sh) {
  while (low < high) {
    const uint64_t mid = low + ((high - low) >> 1) + 1;
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    int mine = 0;
    each_element<F, THREADS>(row, p0, p1, edges, [&](float v, int64_t i) { mine += top_key(v, i) >= mid ? 1 : 0; });
    if (mine) atomicAdd(&sh.count, mine);
    __syncthreads();
    const int n = sh.count;
    if (n >= K) {
      low = mid;
      if (n <= kCandidates) break;
    } else {
      high = mid - 1;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  each_element<F, THREADS>(row, p0, p1, edges, [&](float v, int64_t i) {
    const uint64_t key = top_key(v, i);
    if (key >= low) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCandidates) sh.key[at] = key;
    }
  });
  __syncthreads();
}

// Calls out(rank, key) for the K largest of sh's candidates, rank 0 the
// largest.  They arrived in any order; their keys alone decide.
template <int THREADS, class Out>
__device__ __forceinline__ void top_ranked(const TopShared& sh, int K, const Out& out) {
  const int n = sh.count < kCandidates ? sh.count : kCandidates;
  for (int i = (int)threadIdx.x; i < n; i += THREADS) {
    const uint64_t key = sh.key[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += sh.key[j] > key ? 1 : 0;
    if (rank < K) out(rank, key);
  }
}

}  // namespace logits
}  // namespace qlora
