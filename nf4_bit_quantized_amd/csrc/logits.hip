// Log probabilities of given tokens, with the entropy and the most likely
// tokens of the row, and the distillation loss against a teacher's top logits.
//
// With q = softmax(scale * z) over a row of logits z, M = max z:
//   S = sum exp(scale (z - M)),  log q_j = scale (z_j - M) - log S
//   H = log S - sum exp(scale (z - M)) scale (z - M) / S
// One pass over the row: each thread keeps its largest element and, relative to
// R, at most two below its largest y = c z, c = fl32(scale * log2(e)), the sum of
// 2^(y - R) and for H of 2^(y - R) (y - R).  y - R is one FMA, rounded once; up
// to 32 terms are added in 32 bits, in four chains, and the rest in 64; and the
// workgroup's result is brought from R to c M in 64 bits with the same c.
// What matters is a row that is sure of its token, where log S and H are small:
// an element far above the others becomes R itself, so its term, all of S but
// that little, is put right to 64 bits at the end.
//
// A logit of -inf has probability 0.  A row of nothing else has M = -inf,
// log S = -inf: log probabilities -inf, entropy 0.  NaN or +inf in a row makes
// the row's results NaN.  Where |c M| >= 2^24, R is no longer exact enough and
// the row is read a second time with z - M formed first: so masks of the type's
// lowest value, rows of nothing else among them, give their probabilities too.
//
// Bound by HBM and, near it, by the vector units: five instructions to an
// element, one of them an exponential that takes four times an ordinary one's
// cycles, keep the units busy for 78% of the time (88% with alternatives).  4096
// x 128256 bf16 (1.05 GB): 155 us, 6.8 TB/s; 2048 x 128256 82 us, with 64
// alternatives 96; with the entropy, two more instructions to an element, 100.
// One row of 128256 9.0 us, of it 3.4 the units of its one CU, 13 with twenty
// alternatives.  More rows in flight or pieces to a thread change one row's time
// by under 5%; cutting a row over several CUs would take a second launch, whose
// 2.7 us of host time a call of 12 does not get back (a captured one might).
//
// Of a row of 32000 that is sure of its token, log S is off by 7e-8 rms; the
// same sums in one chain of 32 bits, with R up to 32 below the largest y, have
// 3e-7.  Four chains joined in 64 bits have 5e-8, and take 93 us where these take
// 82 (2048 x 128256).
#include <type_traits>

#include "logits.hpp"
#include "logits_top.hpp"
#include "trace.hpp"
#include "wave.hpp"

namespace qlora {
namespace {

using namespace logits;

constexpr float kFar = 1.329227995784916e36f;  // 2^120

// How far a thread's largest y may be above its R, the y of another of its
// elements: that one is then at least 2^-2 of the largest, and S at least 1.25.
constexpr float kAbove = 2.0f;

struct Sums {
  float m = -kMost, R = -kFar;
  double s = 0.0, t = 0.0;
};

// A sum that has left the range came from logits with |y| above 2^24, where R is
// not near enough to y for 2^(y - R) to be small (masks of -1e10, say): next to
// an R that matters it is nothing.  (If there is none, or +inf in the row, the
// row is read a second time.)  NaN stays.
__device__ __forceinline__ double in_range(double s) { return s > (double)kMost ? 0.0 : s; }

// Adds N elements; returns the largest of them.
template <int N, bool ENT>
__device__ __forceinline__ float add(Sums& a, const float (&f)[N], float c) {
  float g = f[0];
#pragma unroll
  for (int e = 1; e < N; ++e) g = fmaxf(g, f[e]);
  a.m = fmaxf(a.m, g);
  const float y = g * c;
  if (y > a.R + kAbove) {
    const float R = fminf(y, kFar), d = a.R - R, k = __builtin_amdgcn_exp2f(d);
    if constexpr (ENT) a.t = k > 0.0f ? (a.t + a.s * d) * k : 0.0;
    a.s = in_range(a.s) * k;
    a.R = R;
  }
  constexpr int C = N < 4 ? N : 4;
  float s[C], t[C];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float d = __builtin_fmaf(f[e], c, -a.R), x = __builtin_amdgcn_exp2f(d);
    s[e % C] = e < C ? x : s[e % C] + x;
    if constexpr (ENT) {  // 0 * -inf stays 0
      const float b = fmaxf(d, -kFar);
      t[e % C] = e < C ? x * b : __builtin_fmaf(x, b, t[e % C]);
    }
  }
#pragma unroll
  for (int w = 1; w < C; w *= 2)
#pragma unroll
    for (int i = 0; i + w < C; i += 2 * w) {
      s[i] += s[i + w];
      if constexpr (ENT) t[i] += t[i + w];
    }
  a.s += (double)s[0];
  if constexpr (ENT) a.t += (double)t[0];
  return g;
}

// The tokens of a teacher's list: bit b of byte p - first stands for element b
// of piece p, in a window of kWindow pieces.
constexpr int kWindow = 8192;

// U pieces to a thread at a time, all loads of a round before the first use;
// the last round loads no further than the row.  seen (or null) receives the
// largest of every span of rounds.
template <int F, bool ENT, bool MASK, int THREADS, int U, bool PAST>
__device__ __forceinline__ void sweep(Sums& a, const Row<F>& row, int p0, int p1, float c, const uint8_t* mask, int first,
                                      TopSeen<THREADS>* seen) {
  constexpr int E = kPer<F>, N = U < 4 ? U : 4;
  const Spans spans = seen ? top_spans<THREADS, U>(p1 - p0) : Spans{0, 1};
  const int shift = spans.shift;
  const bool note = spans.count > 1;
  int rounds = 0;
  float span = kNone;
  const auto round = [&](int p, auto all) {
    if ((rounds & ((1 << shift) - 1)) == 0) span = kNone;
    u32x4_t w[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (all.value || p + u * THREADS < p1) w[u] = row.template load<PAST>(p + u * THREADS);
#pragma unroll
    for (int v = 0; v < U; v += N) {
      if (!all.value && p + v * THREADS >= p1) break;
      float f[N * E];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const bool in = all.value || p + (u + v) * THREADS < p1;
        unpack<F>(w[u + v], f + u * E);
        const uint32_t b = !in ? 0xFFu : MASK ? mask[p + (u + v) * THREADS - first] : 0u;
        if ((MASK || !all.value) && b) {
#pragma unroll
          for (int e = 0; e < E; ++e) f[u * E + e] = (b >> e) & 1u ? kNone : f[u * E + e];
        }
      }
      span = fmaxf(span, add<N * E, ENT>(a, f, c));
    }
    if (note) seen->key[rounds >> shift][threadIdx.x] = (uint16_t)(ordered(span) >> 16);
    ++rounds;
  };
  int p = p0 + (int)threadIdx.x;
  for (; p + (U - 1) * THREADS < p1; p += U * THREADS) round(p, std::true_type());
  if (p < p1) round(p, std::false_type());
  if (note)
    for (int left = (rounds + (1 << shift) - 1) >> shift; left < spans.count; ++left) seen->key[left][threadIdx.x] = 0;
}

struct Reduced {
  float m[16];
  double s[16], t[16];
};

// What a row comes to: M, S and T = sum e log2(e) with
// e = 2^(c (z - M)).
struct Stats {
  float M;
  double S, T;
};

template <int THREADS>
__device__ __forceinline__ float block_max(float m, Reduced& sh) {
  m = wave::largest(m);
  if ((threadIdx.x & 63) == 0) sh.m[threadIdx.x >> 6] = m;
  __syncthreads();
  float v = sh.m[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = fmaxf(v, sh.m[w]);
  return v;
}

template <bool ENT, int THREADS>
__device__ __forceinline__ void block_sum(double s, double t, Reduced& sh, double& S, double& T) {
  s = wave::sum(s);
  if constexpr (ENT) t = wave::sum(t);
  if ((threadIdx.x & 63) == 0) {
    sh.s[threadIdx.x >> 6] = s;
    if constexpr (ENT) sh.t[threadIdx.x >> 6] = t;
  }
  __syncthreads();
  S = T = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    S += sh.s[w];
    if constexpr (ENT) T += sh.t[w];
  }
}

// The statistics of the row; every thread gets them.  With MASK the k elements of
// ids (LDS) are left out.
template <int F, bool ENT, bool MASK, int THREADS, int U, bool PAST>
__device__ Stats statistics(const Row<F>& row, float c, const int64_t* ids, int k,
                            uint32_t* mask, Reduced& sh, float* most = nullptr,
                            TopSeen<THREADS>* seen = nullptr) {
  constexpr int E = kPer<F>;
  const auto listed = [&](int64_t i) {
    bool hit = false;
    if constexpr (MASK)
      for (int j = 0; j < k; ++j) hit |= ids[j] == i;
    return hit;
  };
  const auto pass = [&](const auto& body) {
    const int p0 = row.full0, p1 = row.full1;
    for (int q0 = p0; q0 < p1; q0 += MASK ? kWindow : p1 - p0) {
      const int q1 = MASK && p1 - q0 > kWindow ? q0 + kWindow : p1;
      if constexpr (MASK) {
        __syncthreads();
        for (int w = (int)threadIdx.x; w < kWindow / 4; w += THREADS) mask[w] = 0u;
        __syncthreads();
        if ((int)threadIdx.x < k) {
          const int64_t id = ids[threadIdx.x];
          if (id >= 0 && id < row.vocab) {
            const int64_t at = id + row.head, p = at / E;
            if (p >= q0 && p < q1) atomicOr(&mask[(p - q0) >> 2], 1u << (8 * ((p - q0) & 3) + (int)(at - p * E)));
          }
        }
        __syncthreads();
      }
      body(q0, q1);
    }
  };
  Sums a;
  pass([&](int q0, int q1) { sweep<F, ENT, MASK, THREADS, U, PAST>(a, row, q0, q1, c, reinterpret_cast<const uint8_t*>(mask), q0, seen); });
  const int mine = (int)threadIdx.x < row.edges() ? row.edge((int)threadIdx.x) : -1;
  const float z_edge = mine >= 0 && !listed(mine) ? row.at(mine) : kNone;
  {
    const float f[1] = {z_edge};
    if (mine >= 0) add<1, ENT>(a, f, c);
  }
  if (most) *most = a.m;
  Stats r;
  r.M = block_max<THREADS>(a.m, sh);
  const float y = r.M * c;
  if (!(fabsf(y) < 16777216.0f)) {
    double s = 0.0, t = 0.0;
    const auto one = [&](float z) {
      const float d = (z - r.M) * c, x = __builtin_amdgcn_exp2f(d);
      s += (double)x;
      if constexpr (ENT) t += (double)(x * fmaxf(d, -kFar));
    };
    pass([&](int q0, int q1) {
      for (int p = q0 + (int)threadIdx.x; p < q1; p += THREADS) {
        float f[E];
        unpack<F>(row.load(p), f);
        uint32_t b = 0;
        if constexpr (MASK) b = reinterpret_cast<const uint8_t*>(mask)[p - q0];
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!((b >> e) & 1u)) one(f[e]);
      }
    });
    if (mine >= 0) one(z_edge);
    block_sum<ENT, THREADS>(s, t, sh, r.S, r.T);
  } else {
    if (a.m == r.M) {
      // 2^u in 64 bits in the place of the rounded one; u is what the product rounded, so two terms are enough
      const float u = __builtin_fmaf(r.M, c, -a.R);
      if (fabsf(u) < 0x1p-10f) {
        const double l = 0.6931471805599453 * (double)u;
        a.s += 1.0 + l + 0.5 * l * l - (double)__builtin_amdgcn_exp2f(u);
      }
    }
    const float d = a.R - y, k2 = __builtin_amdgcn_exp2f(d);
    block_sum<ENT, THREADS>(in_range(a.s) * k2, ENT && k2 > 0.0f ? (a.t + a.s * d) * k2 : 0.0, sh, r.S, r.T);
    const double off = (double)y - (double)c * (double)r.M, f = exp2(off);
    if constexpr (ENT) r.T = (r.T + r.S * off) * f;
    r.S *= f;
  }
  if (r.S == 0.0) r.M = kNone;
  return r;
}

// log q of a logit
__device__ __forceinline__ float log_q(float z, float M, double scale, double log_s) {
  if (M == kNone) return kNone;
  return (float)(scale * ((double)z - (double)M) - log_s);
}

// With 1024 threads 64 registers each, so that two rows share a CU: 2048 x 128256
// with the entropy 100 us against 107.  512 threads are faster with the 66 they
// take then (4096 x 32000: 58 against 60).
template <int F, bool ENT, int THREADS, int U, bool PAST>
__global__ __launch_bounds__(THREADS, THREADS == 1024 ? 8 : 1) void k_score(ScoreParams P, float c) {
  __shared__ Reduced red;
  __shared__ TopShared<THREADS> sh_top;
  __shared__ TopSeen<THREADS> seen;
  const int64_t t = blockIdx.x;
  const Row<F> row(P.in.z, t, P.in.ld, (int)P.in.vocab);
  // the given tokens' logits come with the row's first pieces, not behind its last
  const int mine = (int)threadIdx.x;
  const int64_t id = mine < P.n ? P.tokens[t * P.n + mine] : -1;
  const bool given = id >= 0 && id < P.in.vocab;
  const float z = given ? row.at(id) : 0.0f;
  float most;
  const Stats r = statistics<F, ENT, false, THREADS, U, PAST>(row, c, nullptr, 0, nullptr, red, &most, P.top ? &seen : nullptr);
  const double log_s = log(r.S), scale = (double)P.in.scale;
  if (mine < P.n) P.logprob[t * P.n + mine] = given ? log_q(z, r.M, scale, log_s) : 0.0f;
  if (threadIdx.x == 0) {
    P.stats[2 * t] = r.M;
    P.stats[2 * t + 1] = (float)log_s;
    if constexpr (ENT) P.entropy[t] = r.S == 0.0 ? 0.0f : (float)(log_s - 0.6931471805599453 * (r.T / r.S));
  }
  if (P.top > 0) {
    top_candidates<F, THREADS, U>(row, P.top, most, seen, sh_top);
    top_ranked<THREADS>(sh_top.key, sh_top.count, P.top, [&](int rank, uint64_t key) {
      P.top_ids[t * P.top + rank] = top_index(key);
      P.top_logprob[t * P.top + rank] = log_q(top_value(key), r.M, scale, log_s);
    });
  }
}

// The loss of a row from the statistics of its elements (with REST, of those
// that are not in the teacher's list), by one wave with two entries to a lane.
// Everything is in 64 bits: the loss is a small difference of large terms.
//   rest == 0: p = softmax(values);  loss = sum p (log p - log q)
//   rest == 1: p = exp(values), left = max(0, 1 - sum p), and with q_r the
//     probability outside the list  loss += left (log left - log q_r)
// stats: M, log S, and what the gradient scale * (whole q - p) takes: `whole`
// for the listed tokens, whole - ratio for the others (ratio = left / q_r).
// Entries outside 0 .. vocab - 1 are left out; with none left, whole = 0.  Where
// q_r = 0 the bucket is left out.
struct Listed {  // two entries of a lane
  int64_t id[2];
  bool in[2];
  float v[2], z[2];
};

template <bool REST>
__device__ void distill_finish(const DistillParams& P, int64_t t, const Listed& list, const int64_t* ids, Stats r) {
  const int lane = (int)threadIdx.x;
  const double scale = (double)P.in.scale;
  const auto& in = list.in;
  const auto& z = list.z;
  double v[2] = {(double)list.v[0], (double)list.v[1]};
  const bool any = __ballot(in[0] || in[1]) != 0;
  double known = 0.0, log_known = 0.0;
  if constexpr (!REST) {
    const double most = (double)wave::largest(fmaxf(list.v[0], list.v[1]));
    if (most > -__builtin_inf()) {
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] -= most;
      known = wave::sum(exp(v[0]) + exp(v[1]));
      log_known = log(known);
    }
  } else {
    known = wave::sum(exp(v[0]) + exp(v[1]));
    // the listed elements join the sum, each token once
    bool first[2] = {in[0], in[1]};
    for (int j = 0; j < P.k; ++j) {
      const int64_t other = ids[j];
      first[0] = first[0] && !(j < lane && other == list.id[0]);
      first[1] = first[1] && !(j < lane + 64 && other == list.id[1]);
    }
    const float most = fmaxf(r.M, wave::largest(fmaxf(z[0], z[1])));
    if (most > kNone) {
      double s = 0.0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (first[h]) s += exp(scale * ((double)z[h] - (double)most));
      s = wave::sum(s);
      r.S *= r.S == 0.0 ? 0.0 : exp(scale * ((double)r.M - (double)most));
      r.M = most;
      r.T = r.S;  // the sum outside the list
      r.S += s;
    } else {
      r.T = r.S;
      if (__ballot(z[0] != z[0] || z[1] != z[1])) {  // nothing but NaN, which no comparison shows
        r.S = __builtin_nan("");
        r.M = __builtin_nanf("");
      }
    }
  }
  const double log_s = log(r.S);
  double loss = 0.0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const double lp = v[h] - log_known, p = exp(lp);
    if (p > 0.0) loss += p * (lp - (scale * ((double)z[h] - (double)r.M) - log_s));
  }
  loss = wave::sum(loss);
  double whole = any && known > 0.0 ? 1.0 : 0.0, ratio = 0.0;
  if constexpr (REST) {
    whole = known;
    const double left = 1.0 - known;
    if (any && left > 0.0 && r.T > 0.0) {
      const double q_r = r.T / r.S;
      loss += left * (log(left) - log(q_r));
      ratio = left / q_r;
      whole = 1.0;
    }
  }
  if (r.S == 0.0) loss = whole > 0.0 ? __builtin_inf() : 0.0;
  if (r.S != r.S && any) loss = r.S;
  if (lane == 0) {
    P.loss[t] = (float)loss;
    P.stats[4 * t] = r.M;
    P.stats[4 * t + 1] = (float)log_s;
    P.stats[4 * t + 2] = (float)whole;
    P.stats[4 * t + 3] = (float)fmin(ratio, 1e30);
  }
}

template <int F, bool REST, int THREADS, int U, bool PAST>
__global__ __launch_bounds__(THREADS) void k_distill(DistillParams P, float c) {
  __shared__ Reduced red;
  __shared__ uint32_t mask[REST ? kWindow / 4 : 1];
  __shared__ int64_t ids[REST ? kLogitsMost : 1];
  const int64_t t = blockIdx.x;
  const Row<F> row(P.in.z, t, P.in.ld, (int)P.in.vocab);
  // the entries and their logits come with the row's first pieces, not behind its last
  Listed list;
  if (threadIdx.x < 64) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = (int)threadIdx.x + 64 * h;
      list.id[h] = i < P.k ? P.ids[t * P.k + i] : -1;
      list.in[h] = list.id[h] >= 0 && list.id[h] < P.in.vocab;
      list.v[h] = list.in[h] ? P.values[t * P.k + i] : kNone;
      list.z[h] = list.in[h] ? row.at(list.id[h]) : kNone;
      if (REST && i < P.k) ids[i] = list.id[h];
    }
  }
  if constexpr (REST) __syncthreads();
  const Stats r = statistics<F, false, REST, THREADS, U, PAST>(row, c, ids, P.k, mask, red);
  if (threadIdx.x < 64) distill_finish<REST>(P, t, list, ids, r);
}

float log2_scale(float scale) { return (float)((double)scale * 1.4426950408889634); }

// Threads to a row, from the row's bytes and the number of rows.  A thread
// takes four pieces of 16 bytes at a time, so 256, 512 or 1024 threads want
// 16, 32 or 64 KB of row a round, and what a last round leaves idle counts.  us
// with 256, 512 and 1024 threads (statistics and one log probability, bf16,
// without the entropy, which goes by the same rule):
//   4096 x 16000   28.5  30.3  48.8        2048 x 64000   47.8  47.4  44.9
//   4096 x 32000   49.3  47.3  62.7        2048 x 128256  89.9  89.5  85.4
//   4096 x 50257   73.9  70.7  77.5        77 x 50257 (fp32, five alternatives)  14.4  9.5  12.1
// Up to one row to a CU, 512 are faster than 1024 at any length.
int row_threads(int64_t T, int64_t bytes) {
  if (bytes < 48 << 10) return 256;
  return T <= 256 || bytes < 112 << 10 ? 512 : 1024;
}

template <class Go>
void by_format(int format, const Go& go) {
  if (format == kWeightF32) go(std::integral_constant<int, kWeightF32>());
  else if (format == kWeightBf16) go(std::integral_constant<int, kWeightBf16>());
  else go(std::integral_constant<int, kWeightF16>());
}

// 4096 x 128256 bf16 (1.05 GB) after their gradients were written: 154 us past
// the caches, 174 through them; 2048 x 128256 80 and 86, with 64 alternatives
// (which read some pieces twice) 94 and 98.
bool read_past(const LogitsRows& in) { return in.T * in.bytes() >= kCacheBytes; }

}  // namespace

template <int N>
using Int = std::integral_constant<int, N>;

hipError_t launch_score(const ScoreParams& P, hipStream_t stream) {
  if (P.in.T == 0) return hipSuccess;
  const float c = log2_scale(P.in.scale);
  const int threads = row_threads(P.in.T, P.in.bytes());
  by_format(P.in.format, [&](auto f) {
    const auto go = [&](auto n, auto past) {
      constexpr int F = decltype(f)::value, N = decltype(n)::value;
      constexpr bool PAST = decltype(past)::value;
      const dim3 grid((unsigned)P.in.T), block(N);
      if (P.entropy) launch(KID_LOGPROB, k_score<F, true, N, 4, PAST>, grid, block, stream, P, c);
      else launch(KID_LOGPROB, k_score<F, false, N, 4, PAST>, grid, block, stream, P, c);
    };
    const auto by_threads = [&](auto past) {
      if (threads == 256) go(Int<256>(), past);
      else if (threads == 512) go(Int<512>(), past);
      else go(Int<1024>(), past);
    };
    if (read_past(P.in)) by_threads(std::true_type());
    else by_threads(std::false_type());
  });
  return hipGetLastError();
}

hipError_t launch_distill(const DistillParams& P, hipStream_t stream) {
  if (P.in.T == 0) return hipSuccess;
  const float c = log2_scale(P.in.scale);
  const int64_t bytes = P.in.bytes();
  const int threads = row_threads(P.in.T, bytes);
  by_format(P.in.format, [&](auto f) {
    const auto go = [&](auto rest, auto n, auto u, auto past) {
      constexpr int F = decltype(f)::value, N = decltype(n)::value, U = decltype(u)::value;
      launch(KID_DISTILL, k_distill<F, decltype(rest)::value, N, U, decltype(past)::value>, dim3((unsigned)P.in.T), dim3(N),
             stream, P, c);
    };
    const auto by_threads = [&](auto past) {
      if (P.rest) {
        // the mask costs barriers, which small workgroups feel less.  us with 256 threads and four or eight pieces,
        // 512 and 1024 with four: 4096 x 32000 55.0 63.4 70.9 108; 2048 x 64000 54.3 51.5 54.5 69.7; 2048 x 128256
        // 102 96 97 111.  Few rows: 77 x 50257 (fp32) 19.1 16.2 14.2 15.6.
        if (P.in.T <= 256 && threads >= 512) go(std::true_type(), Int<512>(), Int<4>(), past);
        else if (bytes < 112 << 10) go(std::true_type(), Int<256>(), Int<4>(), past);
        else go(std::true_type(), Int<256>(), Int<8>(), past);
      } else if (threads == 256) {
        go(std::false_type(), Int<256>(), Int<4>(), past);
      } else if (threads == 512) {
        go(std::false_type(), Int<512>(), Int<4>(), past);
      } else {
        go(std::false_type(), Int<1024>(), Int<4>(), past);
      }
    };
    if (read_past(P.in)) by_threads(std::true_type());
    else by_threads(std::false_type());
  });
  return hipGetLastError();
}

}  // namespace qlora
