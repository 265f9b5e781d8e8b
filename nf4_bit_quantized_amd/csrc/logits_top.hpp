// The largest elements of a row, ties to the lower index.
//
// An element's key is its value in the order of the floats (32 bits), then its
// index from the end (32 bits): no two are alike, so "the k largest" is one set
// in one order whatever the ties.
#pragma once

#include <type_traits>

#include "logits.hpp"

namespace qlora {
namespace logits {

constexpr int kCandidates = 1024;

__device__ __forceinline__ uint64_t top_key(float v, int64_t i) {
  return ((uint64_t)ordered(v) << 32) | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ int64_t top_index(uint64_t key) { return (int64_t)(0xFFFFFFFFu - (uint32_t)key); }
__device__ __forceinline__ float top_value(uint64_t key) { return from_ordered((uint32_t)(key >> 32)); }

// What a thread has seen of a row, in kSpans spans of 2^shift rounds of U pieces:
// the first 16 bits of the key of each span's largest element.
constexpr int kSpans = 8;
template <int THREADS>
struct TopSeen {
  uint16_t key[kSpans][THREADS];
};

template <int THREADS>
struct TopShared {
  uint64_t key[kCandidates];
  uint32_t most[256];               // keys of the groups of threads
  uint16_t who[kSpans * THREADS];   // threads, and their spans from bit 10 on, that hold candidates
  int count, holders;
  uint32_t low, below, above;
};

// One round is one span, and that the thread's `most`.
struct Spans {
  int shift, count;
};
template <int THREADS, int U>
__device__ __forceinline__ Spans top_spans(int pieces) {
  const int rounds = (pieces + U * THREADS - 1) / (U * THREADS);
  if (rounds <= 1) return Spans{0, 1};
  int shift = 0;
  while ((rounds - 1) >> shift >= kSpans) ++shift;
  return Spans{shift, ((rounds - 1) >> shift) + 1};
}

// A limit that at least K of the wave's 256 keys reach: exactly K, or the K-th
// largest with its last 16 bits cleared; 0 if it has fewer than K above 0.  Bit
// by bit from the top.
__device__ __forceinline__ uint32_t top_limit(const uint32_t (&key)[4], int K) {
  uint32_t t = 0;
  for (int b = 31; b >= 16; --b) {
    const uint32_t next = t | (1u << b);
    int n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) n += __popcll(__ballot(key[j] >= next));
    if (n >= K) t = next;
    if (n == K) break;
  }
  return t;
}

// Calls at(value, index) for every element of the row.
template <int F, int THREADS, class At>
__device__ __forceinline__ void each_element(const Row<F>& row, const At& at) {
  for (int p = row.full0 + (int)threadIdx.x; p < row.full1; p += THREADS) {
    float f[kPer<F>];
    unpack<F>(row.load(p), f);
    const int64_t i0 = (int64_t)p * kPer<F> - row.head;
#pragma unroll
    for (int e = 0; e < kPer<F>; ++e) at(f[e], i0 + e);
  }
  if ((int)threadIdx.x < row.edges()) {
    const int i = row.edge((int)threadIdx.x);
    at(row.at(i), (int64_t)i);
  }
}

// Puts the K largest elements of the row into sh.key, whatever their ties; `low` is at most the first 32 bits of the K-th largest's key.
// First the K-th largest value: how many are above a value between the bounds
// says on which side of it the K-th is, and the nearest elements on both sides
// of it are the new bounds, so a row of few values is decided in as many passes
// and any row in 33: the first value, the end of the limit's own 2^16, may leave
// out as few as those, and each later one halves what is left.  Then, in two
// more, all above it, and as many equal to it as are left, in the order of
// their indexes.
template <int F, int THREADS>
__device__ void top_exact(const Row<F>& row, int K, uint32_t low, TopShared<THREADS>& sh) {
  uint32_t high = 0xFFFFFFFFu, mid = low | 0xFFFFu;
  while (low < high) {
    __syncthreads();
    if (threadIdx.x == 0) {
      sh.count = 0;
      sh.below = 0u;
      sh.above = 0xFFFFFFFFu;
    }
    __syncthreads();
    int n = 0;
    uint32_t below = 0u, above = 0xFFFFFFFFu;
    each_element<F, THREADS>(row, [&](float v, int64_t) {
      const uint32_t k = ordered(v);
      if (k > mid) {
        ++n;
        above = k < above ? k : above;
      } else {
        below = k > below ? k : below;
      }
    });
    if (n) atomicAdd(&sh.count, n);
    atomicMax(&sh.below, below);
    atomicMin(&sh.above, above);
    __syncthreads();
    if (sh.count >= K) low = sh.above;
    else high = sh.below > low ? sh.below : low;
    mid = low + (high - low) / 2;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  each_element<F, THREADS>(row, [&](float v, int64_t i) {
    if (ordered(v) > low) sh.key[atomicAdd(&sh.count, 1)] = top_key(v, i);  // fewer than K
  });
  __syncthreads();
  int left = K - sh.count;
  // one step along the row: a thread's N elements from index i0 on, of which those in [0, vocab) count
  const auto step = [&](auto size, const float* f, int64_t i0, bool in) {
    constexpr int N = decltype(size)::value;
    int mine = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) mine += in && ordered(f[e]) == low ? 1 : 0;
    int before = mine;  // of this wave's lanes up to this one
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int x = __shfl_up(before, o, 64);
      if ((int)(threadIdx.x & 63) >= o) before += x;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) sh.most[threadIdx.x >> 6] = (uint32_t)before;
    __syncthreads();
    before -= mine;
    int all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < (int)(threadIdx.x >> 6)) before += (int)sh.most[w];
      all += (int)sh.most[w];
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (in && ordered(f[e]) == low && before++ < left) sh.key[atomicAdd(&sh.count, 1)] = top_key(f[e], i0 + e);
    left -= all;
  };
  const auto edge = [&](int q0, int q1) {
    const int q = q0 + (int)threadIdx.x;
    const float f[1] = {q < q1 ? row.at(row.edge(q)) : 0.0f};
    step(std::integral_constant<int, 1>(), f, q < q1 ? row.edge(q) : 0, q < q1);
  };
  edge(0, row.edge0());
  for (int p = row.full0; p < row.full1 && left > 0; p += THREADS) {
    const int mine = p + (int)threadIdx.x;
    const bool in = mine < row.full1;
    float f[kPer<F>];
    unpack<F>(row.load(in ? mine : p), f);
    step(std::integral_constant<int, kPer<F>>(), f, (int64_t)mine * kPer<F> - row.head, in);
  }
  if (left > 0) edge(row.edge0(), row.edges());
  __syncthreads();
}

// The same with a pass over few pieces: `most` is the largest element that this
// thread has read, of the full pieces every THREADS-th and at most one edge,
// never above it and at least -kMost.  Of 256 groups of threads, K have their
// largest element at or above the limit; so K elements are, and whatever is lies
// in a thread's span whose largest is: those spans alone are read again.  They
// come from HBM, a line of 128 bytes for each piece of 16, so what counts is how
// few.  Of 2048 x 128256 logits the 64 largest of each row take 95 us (80 without
// them, 112 where all of a thread's pieces are read again), 20 take 88; of 4096
// x 32000, 67 (47, 69) and 57.
// Rows of many like elements overflow the candidates and take the way above.
template <int F, int THREADS, int U>
__device__ void top_candidates(const Row<F>& row, int K, float most, const TopSeen<THREADS>& seen,
                               TopShared<THREADS>& sh) {
  constexpr int G = THREADS / 256;
  const uint32_t mine = most > -kMost ? ordered(most) : 0u;
  uint32_t group = mine;
  if constexpr (G >= 2) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)group, 0xB1, 0xF, 0xF, false);  // lane ^ 1
    group = o > group ? o : group;
  }
  if constexpr (G >= 4) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)group, 0x4E, 0xF, 0xF, false);  // lane ^ 2
    group = o > group ? o : group;
  }
  if ((int)threadIdx.x % G == 0) sh.most[threadIdx.x / G] = group;
  if (threadIdx.x == 0) sh.count = sh.holders = 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    uint32_t key[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) key[j] = sh.most[64 * j + threadIdx.x];
    // the type of the logits decides sixteen bits of a key; for fp32 it is a limit all the same
    const uint32_t low = top_limit(key, K);
    if (threadIdx.x == 0) sh.low = low;
  }
  __syncthreads();
  const uint32_t low = sh.low;
  const Spans spans = top_spans<THREADS, U>(row.full1 - row.full0);
  if (mine >= low) {
    uint32_t held = 1;  // a bit for each span
    if (spans.count > 1) {
      held = 0;
#pragma unroll
      for (int span = 0; span < kSpans; ++span) held |= seen.key[span][threadIdx.x] >= low >> 16 ? 1u << span : 0u;
      held &= (1u << spans.count) - 1;
    }
    int at = atomicAdd(&sh.holders, __popc(held));
    for (; held; held &= held - 1) sh.who[at++] = (uint16_t)(threadIdx.x | (__ffs(held) - 1) << 10);
  }
  __syncthreads();
  const auto offer = [&](float v, int64_t i) {
    const uint32_t k = ordered(v);
    if (k < low) return;
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCandidates) sh.key[at] = ((uint64_t)k << 32) | (0xFFFFFFFFu - (uint32_t)i);
  };
  const int holders = sh.holders, each = U << spans.shift;
  for (int x = (int)threadIdx.x; x < holders * each; x += THREADS) {
    const int j = x / holders, who = (int)sh.who[x - j * holders];
    const int64_t at = (int64_t)row.full0 + (who & 1023) + ((int64_t)(who >> 10) * each + j) * THREADS;
    if (at >= row.full1 || *(volatile int*)&sh.count > kCandidates) continue;
    const int p = (int)at;
    float f[kPer<F>];
    unpack<F>(row.load(p), f);
    const int64_t i0 = (int64_t)p * kPer<F> - row.head;
#pragma unroll
    for (int e = 0; e < kPer<F>; ++e) offer(f[e], i0 + e);
  }
  if ((int)threadIdx.x < row.edges()) {
    const int i = row.edge((int)threadIdx.x);
    offer(row.at(i), (int64_t)i);
  }
  __syncthreads();
  if (sh.count > kCandidates) top_exact<F, THREADS>(row, K, low, sh);
}

// Calls out(rank, key) for the K largest of n keys, rank 0 the largest.  They
// arrived in any order; they alone decide.  Eight lanes to a key, each counting
// the larger among an eighth of the others.
template <int THREADS, class Out>
__device__ __forceinline__ void top_ranked(const uint64_t* keys, int n, int K, const Out& out) {
  for (int i = (int)threadIdx.x >> 3; i < n; i += THREADS / 8) {
    const uint64_t key = keys[i];
    int rank = 0;
    for (int j = (int)threadIdx.x & 7; j < n; j += 8) rank += keys[j] > key ? 1 : 0;
    rank += __builtin_amdgcn_update_dpp(0, rank, 0xB1, 0xF, 0xF, false);   // lane ^ 1
    rank += __builtin_amdgcn_update_dpp(0, rank, 0x4E, 0xF, 0xF, false);   // lane ^ 2
    rank += __builtin_amdgcn_update_dpp(0, rank, 0x141, 0xF, 0xF, false);  // the other four of eight
    if ((threadIdx.x & 7) == 0 && rank < K) out(rank, key);
  }
}

}  // namespace logits
}  // namespace qlora
