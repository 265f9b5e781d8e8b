// Sums of partial results in the order of their ranges.
#pragma once

namespace qlora {

// at(0) + at(1) + ... + at(n - 1), left to right.  The loads go out eight at a
// time (behind the last, it is loaded again and dropped): one by one, each would
// wait for the one before it, about a microsecond where another XCD wrote it.
template <class Load>
__device__ __forceinline__ auto ordered_sum(int n, const Load& at) -> decltype(at(0)) {
  auto v = at(0);
  for (int q0 = 1; q0 < n; q0 += 8) {
    decltype(at(0)) x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = at(q0 + q < n ? q0 + q : n - 1);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q0 + q < n) v += x[q];
  }
  return v;
}

}  // namespace qlora
