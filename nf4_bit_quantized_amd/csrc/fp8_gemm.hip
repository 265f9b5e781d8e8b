// Products of two 8-bit forms (fp8.hip): the base product of a linear layer on
// an 8-bit weight and its input gradient, with the adapter's rank-r term as a
// tail of the same fp32 accumulators:
//   C[t][n] = bf16( sum_k X[t][k] W[n][k] + sum_c At[t][c] Bt[n][c] )
//   C[t][k] = bf16( sum_n X[t][n] W[n][k] + sum_c At[t][c] Bt[k][c] )   (dx)
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 by 64 x 32 codes and both
// operands' scales, half a block of 128: lane l holds row (column) l % 32 and
// 32 consecutive codes, those from 32 (l / 32) of the 64, and its row's scale
// byte.  The first operand is the weight, so four consecutive results of a
// lane are four consecutive output features of one token.
//
// Precision: the unit adds products in groups of eight consecutive codes
// aligned to the group's largest, dropping what lies below 2^-13 of it, and
// everything after that in fp32 (measured: beside a product of 2^8, one of 2^-5
// is kept at each of the 63 other places, one of 2^-6 is lost at the seven of
// the same group and at no other; a test holds the units to the former).  A
// dropped bit is at most 2^-13 of one product, against the 2^-4 that each code
// is already rounded by and the 2^-8 of the result.
//
// Tiles of 256 x 256: one workgroup of four waves per CU, one wave per SIMD
// with 512 registers.  Wave (a, b) owns features 128 a .. +127 and tokens 128 b
// .. +127: 4 x 4 tiles of 32 x 32, 256 fp32 accumulators a lane.  Tiles of 128
// x 128, two workgroups per CU, are half of that each way (plan_product).
//
// What bounds such a tile is how fast operands reach the matrix units, which a
// step of 64 occupies for 1024 cycles at the full rate.  At 4096 x 8192 x 8192
// (one box; TFLOP/s with the outputs of every variant in place):
//   2700  this kernel: both operands copied in rows of 128 bytes
//   2430  copies in rows of 64 bytes: as many bytes, twice the L2 requests
//   2290  the weight's fragments loaded from global memory into registers (a
//         fragment's neighbouring lanes lie in different rows, 64 lookups a load)
//   3060  without the copies and the fragment reads (matrix units, their
//         scales, barriers and the output alone)
// Starting tiles at different places of the contraction costs 2-25%: the 32
// tiles of an XCD live off each other's rows in its L2.
//
// Pipeline, per wave and step u: both operands are copied into a ring of five
// LDS slots, each 128 of the contraction (two steps) of one operand, X two
// pairs of steps ahead and W one and a half; a step's fragments are read
// during the step before it.  The one barrier of a pair stands in its second
// step, behind the second MFMA: by then every wave has waited for its copies
// of the next pair and for its last fragments of this one, whose slots the
// next copies refill.
//
// Rows of a slot are 128 bytes, chunk c of row R at c ^ R % 8 ^ R / 8 % 2: the
// 16 lanes of a fragment read (16 rows, one chunk) fall on distinct bank
// groups.  The weight of dx, whose contraction runs down its rows, is kept as
// [128 rows][256 columns] with piece c of row R at c ^ 2 (R % 8), and read with
// transposing reads (16 lanes: 8 rows of 16 bytes, a lane receives a column).
#include "dma.hpp"
#include "fp8.hpp"
#include "fp8_down.hpp"
#include "fp8_sum.hpp"
#include "fp8_tail.hpp"
#include "trace.hpp"

#include <type_traits>

namespace qlora {
namespace {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef int v2i_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) v2i_t lds_v2i_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;
typedef const __attribute__((address_space(4))) uint32_t* const_u32;

constexpr uint32_t kSlots = 5;

struct WideLaunch {
  Fp8Params p;
  int32_t mt, nt, group;  // token tiles, feature tiles, token tiles walked together
  int32_t f_begin;        // the first feature
  int32_t nsplit;         // contraction ranges of a tile
  uint32_t split_steps;   // steps of a range, a multiple of 8
  int32_t partial;        // the sums go to p.part, [range][T][features]
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf(const void* p, int64_t bytes) {
  const int32_t n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (int32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, 0x00020000);
}

template <int Q>
__device__ __forceinline__ f32x16_t mfma8(v8i_t a, v8i_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, Q, (int)sa, Q, (int)sb);
}

// Eight rows of a lane's column, read transposed.  The pointer is restrict-
// qualified: the slot read is never one that a copy in flight writes (the waits
// and the barrier of each pair see to it), and without the word the compiler
// drains every copy before such a read.
__device__ __forceinline__ v2i_t read_tr8(const uint8_t* __restrict__ slot, uint32_t off) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i_t*)((lds_u8_t*)slot + off));
}

// DX: the weight's contraction runs down its rows; S: 32 x 32 tiles of a wave
// each way (4: tiles of 256 x 256, a workgroup per CU; 2: 128 x 128, two).
template <bool DX, int S>
__device__ __forceinline__ void product(const WideLaunch& L, const uint32_t bid, uint8_t* lds) {
  constexpr int WT = 64 * S, WF = 64 * S;       // tokens and features of the tile
  constexpr uint32_t kSlot = WT * 128;
  constexpr int kLds = kSlots * kSlot;
  constexpr int kOutLd = WF + 8;
  constexpr int M = S * S;                      // MFMAs of a step
  constexpr int NR = 4 * S;                     // its fragment reads
  constexpr int NC = 2 * S;                     // copies of an operand's pair of steps, a wave
  constexpr int BAR = S == 4 ? 1 : 0;           // the barrier's place among the MFMAs
  static_assert(WT * kOutLd * 2 <= kLds, "the output tile fits over the slots");
  struct Frags {
    u32x4_t x[S][2], w[S][2];
  };
  // the n-th slot after the one at byte o
  auto slot_after = [](uint32_t o, uint32_t n) { return o + n * kSlot < kLds ? o + n * kSlot : o + n * kSlot - kLds; };
  const Fp8Params& p = L.p;
  // runs of consecutive tiles go to one XCD; in their order, groups of token
  // tiles are walked feature tile by feature tile
  const uint32_t mt = (uint32_t)L.mt, nt = (uint32_t)L.nt, gm = (uint32_t)L.group;
  const uint32_t run = (mt * nt * (uint32_t)L.nsplit + 7) / 8;
  uint32_t order = bid % 8 * run + bid / 8;
  if (order >= mt * nt * (uint32_t)L.nsplit) return;
  // the ranges of the contraction follow each other, each over all the tiles
  const uint32_t split = __builtin_amdgcn_readfirstlane(order / (mt * nt));
  order -= split * (mt * nt);
  const uint32_t first = order / (gm * nt) * gm;
  const uint32_t rows = mt - first < gm ? mt - first : gm;
  const uint32_t in_group = order - first * nt;
  // (in scalar registers: they go into the buffer resources)
  const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane((first + in_group % rows) * WT);
  const int64_t f0 = (int64_t)__builtin_amdgcn_readfirstlane(L.f_begin + in_group / rows * WF);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wf = 32 * S * (wave & 1), wt = 32 * S * (wave >> 1);
  const int g = lane >> 5, c32 = lane & 31, i16 = lane & 15;
  const int64_t len = DX ? p.Nw : p.Kw, feats = DX ? p.Kw : p.Nw;
  const uint32_t first_step = split * L.split_steps;
  const uint32_t steps_left = (uint32_t)(len / 64) - first_step;
  const uint32_t nsteps = __builtin_amdgcn_readfirstlane(steps_left < L.split_steps ? steps_left : L.split_steps);
  const int64_t k0 = (int64_t)first_step * 64;  // a multiple of 512: whole dwords of scales

  // both operands from the range's first position on
  const int64_t xbase = t0 * len + k0, wbase = DX ? k0 * p.Kw + f0 : f0 * len + k0;
  const int64_t xbytes = (p.T - t0) * len - k0, wbytes = p.Nw * p.Kw - wbase;
  const __amdgpu_buffer_rsrc_t rx = buf(p.X + xbase, xbytes), rw = buf(p.W + wbase, wbytes);
  const __amdgpu_buffer_rsrc_t rs = buf(p.Xs, p.T * fp8_scale_ld(len));

  // copies of a pair of steps: eight kilobytes of each operand a wave.  Rows
  // past the last token or feature read zeros.
  uint32_t xoff[NC], woff[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int R = 16 * S * wave + 8 * j + (lane >> 3);
    const int chunk = (lane & 7) ^ (lane >> 3) ^ (j & 1);
    xoff[j] = t0 + R < p.T ? (uint32_t)(R * len + chunk * 16) : dma::kOob;
    if (DX) {
      const int n = S == 4 ? 32 * wave + 4 * j + (lane >> 4) : 32 * wave + 8 * j + (lane >> 3);
      const int piece = S == 4 ? i16 ^ (2 * (n & 7)) : (lane & 7) ^ (n & 6);
      woff[j] = f0 + piece * 16 < feats ? (uint32_t)(n * p.Kw + piece * 16) : dma::kOob;
    } else {
      woff[j] = f0 + R < feats ? (uint32_t)(R * len + chunk * 16) : dma::kOob;
    }
  }
  const uint32_t wpair = DX ? (uint32_t)(128 * p.Kw) : 128u;
  const uint32_t pairs = (nsteps + 1) / 2;
  // copy j (0 .. NC - 1) of X's or W's pair `pr` into a slot
  auto copy_x = [&](uint32_t pr, uint32_t slot, int j) {
    const uint32_t at = pr < pairs ? pr : pairs - 1;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(lds + slot + kSlot / 4 * wave + 1024 * j), 16, xoff[j], at * 128u, 0, 0);
  };
  auto copy_w = [&](uint32_t pr, uint32_t slot, int j) {
    const uint32_t at = pr < pairs ? pr : pairs - 1;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(lds + slot + kSlot / 4 * wave + 1024 * j), 16, woff[j], at * wpair, 0, 0);
  };

  // scales: a dword holds the bytes of four blocks, eight steps
  const uint32_t groups = (nsteps + 7) / 8;
  uint32_t soff[S];
#pragma unroll
  for (int t = 0; t < S; ++t) {
    const int64_t row = t0 + wt + 32 * t + c32;
    soff[t] = (uint32_t)((row < p.T ? row : p.T - 1) * fp8_scale_ld(len) + k0 / 128);
  }
  auto load_sx = [&](uint32_t gr, int t) {
    return __builtin_amdgcn_raw_buffer_load_b32(rs, soff[t], (gr < groups ? gr : groups - 1) * 4u, 0);
  };
  // the wave's features lie in one block of the weight: its bytes lie in one
  // row of the weight's scales, or, for dx, in one column of them
  const int64_t fb = __builtin_amdgcn_readfirstlane((uint32_t)((f0 + wf < feats ? f0 + wf : f0) / 128));
  const int64_t ldw = fp8_scale_ld(p.Kw);
  const uint8_t* ws = p.Ws + (DX ? k0 / 128 * ldw : k0 / 128);
  struct SwRaw {
    uint32_t v[4];
  };
  auto load_sw = [&](uint32_t gr) {
    const uint32_t at = gr < groups ? gr : groups - 1;
    SwRaw r{};
    if (!DX) {
      r.v[0] = *(const_u32)(ws + fb * ldw + 4 * at);
    } else {
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q)
        r.v[q] = *(const_u32)(ws + (4 * at + q < pairs ? 4 * at + q : pairs - 1) * ldw + (fb & ~3LL));
    }
    return r;
  };
  auto sw_of = [&](const SwRaw& r) -> uint32_t {
    if (!DX) return r.v[0];
    const uint32_t sh = 8 * (uint32_t)(fb & 3);
    return (r.v[0] >> sh & 0xFFu) | (r.v[1] >> sh & 0xFFu) << 8 | (r.v[2] >> sh & 0xFFu) << 16 | (r.v[3] >> sh) << 24;
  };

  // fragment reads of half h of a pair; tile t's are 4096 bytes on (dx: rows
  // 64 h + 8 q are WF (64 h + 8 q) bytes on)
  const int sw = (c32 & 7) ^ ((c32 >> 3) & 1);
  uint32_t xpos[2][2], wpos[S];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) xpos[h][e] = (uint32_t)(c32 * 128 + (((4 * h + 2 * g + e) ^ sw) << 4));
#pragma unroll
  for (int f = 0; f < S; ++f) {
    const int piece = (wf >> 4) + 2 * f + ((lane >> 4) & 1);
    const int swz = S == 4 ? i16 & 14 : (i16 >> 1) & 6;
    wpos[f] = (uint32_t)((32 * g + (i16 >> 1)) * WF + ((piece ^ swz) << 4) + 8 * (i16 & 1));
  }
  auto read_x = [&](Frags& F, uint32_t slot, int h, int t, int e) {
    F.x[t][e] = *reinterpret_cast<const u32x4_t*>(lds + (slot + wt * 128) + xpos[h][e] + 4096 * t);
  };
  auto read_w = [&](Frags& F, uint32_t slot, int h, int f, int e) {
    if (DX) {
#pragma unroll
      for (int q = 2 * e; q < 2 * e + 2; ++q) {
        const v2i_t v = read_tr8(lds + slot, wpos[f] + WF * (64 * h + 8 * q));
        F.w[f][e][2 * (q & 1)] = (uint32_t)v[0];
        F.w[f][e][2 * (q & 1) + 1] = (uint32_t)v[1];
      }
    } else {
      F.w[f][e] = *reinterpret_cast<const u32x4_t*>(lds + (slot + wf * 128) + xpos[h][e] + 4096 * f);
    }
  };
  // read n (0 .. NR - 1) of a step's fragments, in the order the MFMAs need them
  auto read = [&](Frags& F, uint32_t xslot, uint32_t wslot, int h, int n) {
    if (n < 2) read_w(F, wslot, h, 0, n);
    else if (n < 2 + 2 * S) read_x(F, xslot, h, (n - 2) >> 1, n & 1);
    else read_w(F, wslot, h, (n - 2 * S) >> 1, n & 1);
  };

  f32x16_t acc[S][S];  // [feature tile][token tile]
#pragma unroll
  for (int f = 0; f < S; ++f)
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[f][t][v] = 0.0f;

  uint32_t sx[S], sxn[S], swc;
  SwRaw swn;
  Frags F[2];
#pragma unroll
  for (int t = 0; t < S; ++t) sx[t] = sxn[t] = load_sx(0, t);
  swn = load_sw(0);
  swc = sw_of(swn);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int j = 0; j < NC; ++j) copy_x(c, 2 * c * kSlot, j);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NC; ++j) copy_w(c, (2 * c + 1) * kSlot, j);
    __builtin_amdgcn_sched_barrier(0);
  }
  dma::wait_vm<2 * NC>();  // the first pair's copies have landed; the second's went out after them
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int n = 0; n < NR; ++n) read(F[0], 0, kSlot, 0, n);

  uint32_t slot = 0;  // X of the step's pair; W's is the next one
  // step u, J = u % 8; in_loop: the loads of the next group's scales are there
  // to be counted (behind the loop nothing uses them, and they are gone)
  auto step = [&](uint32_t u, auto j_, auto in_loop_) {
    constexpr int J = decltype(j_)::value, Q = J / 2;
    constexpr bool loads = decltype(in_loop_)::value;
    constexpr bool odd = J % 2 != 0;
    Frags& C = F[odd];
    Frags& Nx = F[!odd];
    const uint32_t pr = u / 2;
    // the next step's fragments: the pair's second half, or the next pair's first
    const uint32_t rx_ = odd ? slot_after(slot, 2) : slot, rw_ = odd ? slot_after(slot, 3) : slot_after(slot, 1);
    const uint32_t fill = odd ? slot : slot_after(slot, 4);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int f = m / S, t = m % S;
      const u32x4_t w0 = C.w[f][0], w1 = C.w[f][1], x0 = C.x[t][0], x1 = C.x[t][1];
      acc[f][t] = mfma8<Q>(v8i_t{(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]},
                           v8i_t{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]},
                           acc[f][t], swc, sx[t]);
      // what goes out behind this MFMA: its share of the next step's reads and of the copies
      constexpr int first = odd ? BAR + 1 : 0;
      if (odd && m == BAR) {
        // the next pair's copies have landed (after them went out those of X
        // in the step before, and the scales' loads if that was J = 2), and
        // this wave's fragments of the pair are read
        dma::wait_vm<loads && J == 3 ? NC + S : NC>();
        lds_barrier();
      }
      if (m >= first) {
#pragma unroll
        for (int n = NR * (m - first) / (M - first); n < NR * (m + 1 - first) / (M - first); ++n)
          read(Nx, rx_, rw_, odd ? 0 : 1, n);
#pragma unroll
        for (int n = NC * (m - first) / (M - first); n < NC * (m + 1 - first) / (M - first); ++n) {
          if (odd) copy_w(pr + 2, fill, n);
          else copy_x(pr + 2, fill, n);
        }
      }
      if (loads && J == 2 && m % S == 1) sxn[m / S] = load_sx(u / 8 + 1, m / S);
      if (J == 2 && m == M / 2) swn = load_sw(u / 8 + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (odd) slot = slot_after(slot, 2);
  };
  auto steps8 = [&](uint32_t u) {
    step(u, std::integral_constant<int, 0>(), std::true_type());
    step(u + 1, std::integral_constant<int, 1>(), std::true_type());
    step(u + 2, std::integral_constant<int, 2>(), std::true_type());
    step(u + 3, std::integral_constant<int, 3>(), std::true_type());
    step(u + 4, std::integral_constant<int, 4>(), std::true_type());
    step(u + 5, std::integral_constant<int, 5>(), std::true_type());
    step(u + 6, std::integral_constant<int, 6>(), std::true_type());
    step(u + 7, std::integral_constant<int, 7>(), std::true_type());
    swc = sw_of(swn);
  };
  uint32_t u = 0;
  for (; u + 8 <= nsteps; u += 8) {
    steps8(u);
#pragma unroll
    for (int t = 0; t < S; ++t) sx[t] = sxn[t];
  }
  if (u < nsteps) step(u, std::integral_constant<int, 0>(), std::false_type());
  if (u + 1 < nsteps) step(u + 1, std::integral_constant<int, 1>(), std::false_type());
  if (u + 2 < nsteps) step(u + 2, std::integral_constant<int, 2>(), std::false_type());
  if (u + 3 < nsteps) step(u + 3, std::integral_constant<int, 3>(), std::false_type());
  if (u + 4 < nsteps) step(u + 4, std::integral_constant<int, 4>(), std::false_type());
  if (u + 5 < nsteps) step(u + 5, std::integral_constant<int, 5>(), std::false_type());
  if (u + 6 < nsteps) step(u + 6, std::integral_constant<int, 6>(), std::false_type());

  // (lane numbers formed anew: what is derived from them here need not live
  // through the loop, whose registers are all taken)
  int le = lane;
  asm volatile("" : "+v"(le));
  const int ge = le >> 5, ce = le & 31;
  if (p.r > 0 && split == 0) {
    // the next sixteen columns' fragments are loaded while one's multiply
    bf16x8_t wa[2][S], xb[2][S];
    auto load = [&](int c0, bf16x8_t(&w)[S], bf16x8_t(&x)[S]) {
#pragma unroll
      for (int f = 0; f < S; ++f) w[f] = tail_weight(p, f0 + wf + 32 * f + ce, feats, c0 + 8 * ge);
#pragma unroll
      for (int t = 0; t < S; ++t) x[t] = tail_token(p, t0 + wt + 32 * t + ce, c0 + 8 * ge);
    };
    auto mul = [&](const bf16x8_t(&w)[S], const bf16x8_t(&x)[S]) {
#pragma unroll
      for (int f = 0; f < S; ++f)
#pragma unroll
        for (int t = 0; t < S; ++t)
          acc[f][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[f], x[t], acc[f][t], 0, 0, 0);
    };
    load(0, wa[0], xb[0]);
    for (int c0 = 0; c0 < 2 * p.r; c0 += 32) {  // columns up to ldh, a multiple of 64, are there
      load(c0 + 16, wa[1], xb[1]);
      mul(wa[0], xb[0]);
      if (c0 + 32 < 2 * p.r) load(c0 + 32, wa[0], xb[0]);
      mul(wa[1], xb[1]);
    }
  }

  if (L.partial) {
    dma::wait_vm<0>();  // no copy may land in LDS that is no longer this workgroup's
    float* part = p.part + (int64_t)split * p.T * feats;
#pragma unroll
    for (int t = 0; t < S; ++t) {
      const int64_t tok = t0 + wt + 32 * t + ce;
      if (tok >= p.T) continue;
#pragma unroll
      for (int f = 0; f < S; ++f)
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          const int64_t col = f0 + wf + 32 * f + 2 * v + 4 * ge;
          if (col < feats)
            *reinterpret_cast<f32x4_t*>(part + tok * feats + col) =
                f32x4_t{acc[f][t][v], acc[f][t][v + 1], acc[f][t][v + 2], acc[f][t][v + 3]};
        }
    }
    return;
  }

  // every wave's copies have landed and every fragment is read before the
  // output tile goes over the stages
  dma::wait_vm<0>();
  __syncthreads();
  // lane l, value v: token 32 t + l % 32, feature 8 (v / 4) + 4 (l / 32) + v % 4
  uint16_t* out = reinterpret_cast<uint16_t*>(lds);
#pragma unroll
  for (int f = 0; f < S; ++f)
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
      for (int v = 0; v < 16; v += 4)
        *reinterpret_cast<uint2*>(out + (wt + 32 * t + ce) * kOutLd + wf + 32 * f + 2 * v + 4 * ge) =
            make_uint2(pack_bf16x2(acc[f][t][v], acc[f][t][v + 1]), pack_bf16x2(acc[f][t][v + 2], acc[f][t][v + 3]));
  __syncthreads();
  for (int e = threadIdx.x; e < WT * WF / 8; e += 256) {
    const int R = e / (WF / 8), col = e % (WF / 8) * 8;
    if (t0 + R < p.T && f0 + col < feats)
      *reinterpret_cast<u32x4_t*>(p.C + (t0 + R) * feats + f0 + col) = *reinterpret_cast<const u32x4_t*>(out + R * kOutLd + col);
  }
}

constexpr int kLds256 = kSlots * 256 * 128, kLds128 = kSlots * 128 * 128;

__global__ __launch_bounds__(256, 1) void k_fp8_wide_256(WideLaunch L) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds256];
  product<false, 4>(L, blockIdx.x, lds);
}
__global__ __launch_bounds__(256, 1) void k_fp8_wide_256_dx(WideLaunch L) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds256];
  product<true, 4>(L, blockIdx.x, lds);
}
__global__ __launch_bounds__(256, 2) void k_fp8_wide_128(WideLaunch L) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds128];
  product<false, 2>(L, blockIdx.x, lds);
}
__global__ __launch_bounds__(256, 2) void k_fp8_wide_128_dx(WideLaunch L) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds128];
  product<true, 2>(L, blockIdx.x, lds);
}

// Few tokens.  The product is a stream of the weight, and what costs beside it
// is launches: U = X A^T runs in the same one, its workgroups first, and the
// pass that adds the contraction ranges' partial sums also forms the rank-r
// term from U (or, for dx, from G), in fp32.  One token through 28672 x 8192 at
// r = 64, the weight read from HBM: 50 us (4.8 TB/s), of which the last pass 6;
// with U and the sums in launches of their own 8 more.
struct FewLaunch {
  WideLaunch w;
  Fp8DownParams d;
  float* upart;  // [uranges][T][r]
  int32_t jtiles, uranges, uwgs;  // workgroups of U, rounded up to a multiple of eight
  int32_t chunks, chunks_per_range;
};

__global__ __launch_bounds__(256, 2) void k_fp8_few(FewLaunch L) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds128];
  if (blockIdx.x >= (uint32_t)L.uwgs) {
    product<false, 2>(L.w, blockIdx.x - L.uwgs, lds);
    return;
  }
  const int tiles = (int)((L.d.T + 15) / 16) * L.jtiles;
  const int range = (int)blockIdx.x / tiles, tile = (int)blockIdx.x - range * tiles;
  if (range >= L.uranges) return;
  const int64_t t0 = (int64_t)(tile / L.jtiles) * 16;
  const int j0 = tile % L.jtiles * 16;
  const int c_begin = range * L.chunks_per_range;
  const int c_end = c_begin + L.chunks_per_range < L.chunks ? c_begin + L.chunks_per_range : L.chunks;
  float(*red)[16][17] = reinterpret_cast<float(*)[16][17]>(lds);
  fp8::down_tile<4, 17>(L.d, t0, j0, c_begin, c_end, __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), red);
  __syncthreads();
  const int rr = threadIdx.x >> 4, j = threadIdx.x & 15;
  if (t0 + rr < L.d.T && j0 + j < L.d.r)
    L.upart[((int64_t)range * L.d.T + t0 + rr) * L.d.r + j0 + j] =
        ((red[0][rr][j] + red[1][rr][j]) + red[2][rr][j]) + red[3][rr][j];
}

// C[t][f] = bf16( sum over the ranges of part[q][t][f] + s sum_j V[t][j] M ),
// V being U (its ranges' partial sums added here, and U written) or G, M B[f][j]
// or, for dx, A[j][f].  A workgroup: kFewT tokens, a feature a thread.
constexpr int kFewT = 8, kFewF = 128, kFewQ = 4;
constexpr int kFewMaxRank = 128;

struct FinishLaunch {
  const float* part;
  int32_t nsplit;
  int64_t T, feats;
  const float* V;
  int32_t vranges;
  int32_t r;
  float s;
  const uint16_t* M;
  float* U;  // forward, or null
  uint16_t* C;
};

template <bool DX>
__global__ __launch_bounds__(kFewF) void k_fp8_finish(FinishLaunch L) {
  __shared__ float v[kFewT][kFewMaxRank];
  const int64_t t0 = (int64_t)blockIdx.y * kFewT;
  const int nt = (int)(L.T - t0 < kFewT ? L.T - t0 : kFewT);
  const int r = L.r;
  const int64_t f = (int64_t)blockIdx.x * kFewF + threadIdx.x;
  const int64_t fc = f < L.feats ? f : L.feats - 1;
  // tokens past the last repeat it, and are not stored
  int64_t row[kFewT];
  float part[kFewQ][kFewT];
  const auto load_part = [&](int q0) {
#pragma unroll
    for (int q = 0; q < kFewQ; ++q) {
      const float* src = L.part + (int64_t)(q0 + q < L.nsplit ? q0 + q : L.nsplit - 1) * L.T * L.feats;
#pragma unroll
      for (int t = 0; t < kFewT; ++t) part[q][t] = src[row[t]];
    }
  };
#pragma unroll
  for (int t = 0; t < kFewT; ++t) row[t] = (t0 + (t < nt ? t : nt - 1)) * L.feats + fc;
  load_part(0);
  // M's first columns, 64 of them where its rows can be read 16 bytes at a time
  const bool wide = !DX && r % 8 == 0;
  const int64_t sj = DX ? L.feats : 1;
  const uint16_t* m0 = DX ? L.M + fc : L.M + fc * r;
  u32x4_t mw[8];
  uint16_t mn[16];
  const auto load_m = [&](int j0) {
    if (wide) {
#pragma unroll
      for (int q = 0; q < 8; ++q) mw[q] = *reinterpret_cast<const u32x4_t*>(m0 + (j0 + 8 * q < r ? j0 + 8 * q : r - 8));
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q) mn[q] = m0[(j0 + q < r ? j0 + q : r - 1) * sj];
    }
  };
  load_m(0);
  for (int e = threadIdx.x; e < kFewT * r; e += kFewF) {
    const int t = e / r, j = e - t * r;
    if (t >= nt) {
      v[t][j] = 0.0f;
      continue;
    }
    const float* src = L.V + (t0 + t) * r + j;
    const float u = ordered_sum(L.vranges, [&](int q) { return src[(int64_t)q * L.T * r]; });
    v[t][j] = L.s * u;
    if (L.U && blockIdx.x == 0) L.U[(t0 + t) * r + j] = u;
  }
  __syncthreads();
  if (f >= L.feats) return;
  float acc[kFewT];
#pragma unroll
  for (int t = 0; t < kFewT; ++t) acc[t] = part[0][t];
  for (int q0 = 0;;) {
#pragma unroll
    for (int q = 0; q < kFewQ; ++q)
      if (q0 + q > 0 && q0 + q < L.nsplit) {
#pragma unroll
        for (int t = 0; t < kFewT; ++t) acc[t] += part[q][t];
      }
    q0 += kFewQ;
    if (q0 >= L.nsplit) break;
    load_part(q0);
  }
  const auto add = [&](int j, float m) {
#pragma unroll
    for (int t = 0; t < kFewT; ++t) acc[t] = fmaf(v[t][j], m, acc[t]);
  };
  for (int j0 = 0;;) {
    if (wide) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (j0 + 8 * q < r) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t m = mw[q][h];
            add(j0 + 8 * q + 2 * h, bf16_bits_to_f32(m & 0xFFFFu));
            add(j0 + 8 * q + 2 * h + 1, bf16_bits_to_f32(m >> 16));
          }
        }
      }
      j0 += 64;
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (j0 + q < r) add(j0 + q, bf16_bits_to_f32(mn[q]));
      j0 += 16;
    }
    if (j0 >= r) break;
    load_m(j0);
  }
#pragma unroll
  for (int t = 0; t < kFewT; ++t)
    if (t < nt) L.C[(t0 + t) * L.feats + f] = f32_to_bf16_bits(acc[t]);
}

}  // namespace

namespace {
// The contraction ranges' partial sums in range order, rounded once; four
// consecutive elements a thread.
__global__ __launch_bounds__(256) void k_fp8_sum(const float* __restrict__ part, int nsplit, int64_t n,
                                                 uint16_t* __restrict__ C) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= n) return;
  const f32x4_t v = ordered_sum(nsplit, [&](int q) { return *reinterpret_cast<const f32x4_t*>(part + q * n + e); });
  *reinterpret_cast<uint2*>(C + e) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// How a product is cut: the first `wide` features on 256 x 256 tiles, the
// others on 128 x 128 ones, or all of them on those over nsplit contraction
// ranges (a multiple of eight steps each) whose sums a second launch adds.
//
// Times measured at contractions of 4096 to 11008, in microseconds for n steps
// of 64: a full round of 256 large tiles (one a CU) 0.72 n + 4, one of w tiles
// (0.47 + 0.25 w / 256) n + 3; a round of small ones 0.46 n + 3 for 257 to 512
// (two a CU), 0.29 n + 3 for fewer; a further launch 5; a pass over partial sums
// 3 and their bytes, written and read, at 4 TB/s.  So a large tile is done 1.3
// times as fast for its size where rounds are full (4096 x 8192 x 8192: 202 us
// against 265, the model 192 and 247), and the small ones win where they would
// not be (1333 x 4096 x 4096: 31 against 42).  dX goes by the same times: its
// large tiles take as long (4096 x 8192 x 8192: 195), its small ones up to a
// tenth more (1333 x 4096 x 4096: 34; large ones 44).  With all features on
// large and on small tiles, at 1333, 2048 and 4096 tokens and 4096 to 22016
// features and contractions, what the model picks was the faster of the two or
// faster than both, or within 2% of it (forward) and 5% (dX: 8192 features of a
// contraction of 22016, 1333 tokens, 214 against 205).
struct ProductPlan {
  int64_t wide;
  int32_t nsplit;
  uint32_t split_steps;
};

double large_time(int64_t tiles, int64_t steps) {
  const int64_t rest = tiles % 256;
  return (double)(tiles / 256) * (0.72 * steps + 4) + (rest ? (0.47 + 0.25 * rest / 256) * steps + 3 : 0.0);
}
double small_time(int64_t tiles, int64_t steps) {
  const int64_t rest = tiles % 512;
  return (double)(tiles / 512) * (0.46 * steps + 3) + (rest ? (rest > 256 ? 0.46 : 0.29) * steps + 3 : 0.0);
}

ProductPlan plan_product(int64_t T, int64_t feats, int64_t len, bool few) {
  const int64_t steps = len / 64, groups = (steps + 7) / 8;
  const int64_t mt4 = (T + 255) / 256, nt4 = (feats + 255) / 256, mt2 = (T + 127) / 128;
  const auto small_tiles = [&](int64_t f) { return mt2 * ((f + 127) / 128); };
  ProductPlan best{0, 1, (uint32_t)(groups * 8)};
  if (few) {
    // a stream of the weight: ranges of 2048 (256 KB of it a workgroup), more
    // where those give fewer workgroups than CUs.  One token through 28672 x
    // 8192: 50 us at 4 ranges, 60 at 2, 57 at 8; 16 tokens: 58, 71 and 66; 100
    // through 22016 x 8192: 74 at 4 and at 2, 80 at 8; 77 through 8192 x 8192:
    // 27 at 4, 31 at 8
    int64_t s = (groups + 3) / 4;
    const int64_t fill = (256 + small_tiles(feats) - 1) / small_tiles(feats);
    if (s < fill) s = fill;
    if (s > groups) s = groups;
    if (s > 16) s = 16;
    const int64_t per = (groups + s - 1) / s;
    return ProductPlan{0, (int32_t)((groups + per - 1) / per), (uint32_t)(per * 8)};
  }
  double time = small_time(small_tiles(feats), steps);
  // whole rounds of large tiles, the last features on small ones; or large tiles alone
  for (int64_t rounds = 1;; ++rounds) {
    const int64_t cols = rounds * 256 / mt4 < nt4 ? rounds * 256 / mt4 : nt4;
    if (cols > 0) {
      const int64_t wide = cols * 256 < feats ? cols * 256 : feats;
      const double t = large_time(cols * mt4, steps) + (wide < feats ? 5 + small_time(small_tiles(feats - wide), steps) : 0.0);
      if (t < time) {
        time = t;
        best.wide = wide;
      }
    }
    if (cols == nt4) break;
  }
  for (int64_t s = 2; s <= 16 && s <= groups; ++s) {
    const int64_t per = (groups + s - 1) / s;
    if ((groups + per - 1) / per != s) continue;  // an empty range
    const double t = small_time(small_tiles(feats) * s, per * 8) + 3 + (double)(8 * s) * T * feats / 4e6;
    if (t < time) {
      time = t;
      best = ProductPlan{0, (int32_t)s, (uint32_t)(per * 8)};
    }
  }
  return best;
}

template <int S>
WideLaunch tiles_launch(const Fp8Params& p, int64_t f_begin, int64_t f_end, const ProductPlan& plan) {
  WideLaunch L{};
  L.p = p;
  L.mt = (int32_t)((p.T + 64 * S - 1) / (64 * S));
  L.nt = (int32_t)((f_end - f_begin + 64 * S - 1) / (64 * S));
  L.group = 4;
  L.f_begin = (int32_t)f_begin;
  L.nsplit = plan.nsplit;
  L.split_steps = plan.split_steps;
  L.partial = plan.nsplit > 1;
  return L;
}

WideLaunch small_tiles_launch(const Fp8Params& p, const ProductPlan& plan) {
  return tiles_launch<2>(p, 0, p.dx ? p.Kw : p.Nw, plan);
}

template <int S>
hipError_t launch_tiles(const Fp8Params& p, int64_t f_begin, int64_t f_end, const ProductPlan& plan, hipStream_t stream) {
  if (f_begin >= f_end) return hipSuccess;
  const WideLaunch L = tiles_launch<S>(p, f_begin, f_end, plan);
  const int64_t tiles = (int64_t)L.mt * L.nt * L.nsplit;
  KernelEvents ev(KID_FP8_GEMM);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8));
  const auto k = S == 4 ? (p.dx ? k_fp8_wide_256_dx : k_fp8_wide_256) : (p.dx ? k_fp8_wide_128_dx : k_fp8_wide_128);
  hipExtLaunchKernelGGL(k, grid, dim3(256), 0, stream, ev.start(), ev.stop(), 0, L);
  return hipGetLastError();
}
}  // namespace

namespace {
// Few tokens with a rank-r term go through k_fp8_finish, whatever the ranges.
bool is_few(int64_t T, int r) { return T <= kFp8FewT && r > 0; }

int64_t few_ranges(int64_t T, int64_t K, int r) {
  // U's ranges: as many as give its tiles 64 workgroups, four chunks each at
  // least.  With 16 workgroups one token through 4096 x 4096, r = 16, takes 17.9
  // us against 16.7, with 256 18.1; 16 tokens through 8192 x 28672, r = 64: 58
  // with 16, 60 with 64, 71 with 256 (more partial sums for the last pass)
  const int64_t tiles = (T + 15) / 16 * ((r + 15) / 16), chunks = (K + 127) / 128;
  int64_t s = (64 + tiles - 1) / tiles;
  if (s > chunks / 4) s = chunks / 4;
  if (s < 1) s = 1;
  const int64_t per = (chunks + s - 1) / s;
  return (chunks + per - 1) / per;
}
}  // namespace

size_t fp8_product_part_bytes(int64_t T, int64_t Nw, int64_t Kw, int dx, int r) {
  const int64_t feats = dx ? Kw : Nw;
  const bool few = is_few(T, r);
  const ProductPlan plan = plan_product(T, feats, dx ? Nw : Kw, few);
  size_t n = plan.nsplit > 1 || few ? (size_t)plan.nsplit * T * feats * 4 : 0;
  if (few && !dx) n += (size_t)few_ranges(T, Kw, r) * T * r * 4;
  return n;
}

hipError_t launch_fp8_product(const Fp8Params& p, hipStream_t stream) {
  const int64_t feats = p.dx ? p.Kw : p.Nw;
  const bool few = is_few(p.T, p.r);
  const ProductPlan plan = plan_product(p.T, feats, p.dx ? p.Nw : p.Kw, few);
  const size_t need = fp8_product_part_bytes(p.T, p.Nw, p.Kw, p.dx, p.r);
  if (need > 0 && (!p.part || p.part_bytes < need)) return hipErrorInvalidValue;
  if (few) {
    FewLaunch F{};
    F.w = small_tiles_launch(p, plan);
    F.w.p.r = 0;
    F.w.partial = 1;
    const unsigned tiles = (unsigned)(((int64_t)F.w.mt * F.w.nt * F.w.nsplit + 7) / 8 * 8);
    FinishLaunch E{p.part, plan.nsplit, p.T, feats, p.G, 1, p.r, p.s, p.M, nullptr, p.C};
    {
      KernelEvents ev(KID_FP8_GEMM);
      if (p.dx) {
        hipExtLaunchKernelGGL(k_fp8_wide_128_dx, dim3(tiles), dim3(256), 0, stream, ev.start(), ev.stop(), 0, F.w);
      } else {
        F.d.X = p.X; F.d.Xs = p.Xs; F.d.A = p.A; F.d.T = p.T; F.d.K = p.Kw; F.d.r = p.r;
        F.upart = p.part + (size_t)plan.nsplit * p.T * feats;
        F.jtiles = (p.r + 15) / 16;
        F.uranges = (int32_t)few_ranges(p.T, p.Kw, p.r);
        F.chunks = (int32_t)((p.Kw + 127) / 128);
        F.chunks_per_range = (F.chunks + F.uranges - 1) / F.uranges;
        F.uwgs = (int32_t)(((p.T + 15) / 16 * F.jtiles * F.uranges + 7) / 8 * 8);
        E.V = F.upart;
        E.vranges = F.uranges;
        E.U = p.U;
        hipExtLaunchKernelGGL(k_fp8_few, dim3(F.uwgs + tiles), dim3(256), 0, stream, ev.start(), ev.stop(), 0, F);
      }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    KernelEvents ev(KID_REDUCE);
    const dim3 grid((unsigned)((feats + kFewF - 1) / kFewF), (unsigned)((p.T + kFewT - 1) / kFewT));
    hipExtLaunchKernelGGL(p.dx ? k_fp8_finish<true> : k_fp8_finish<false>, grid, dim3(kFewF), 0, stream, ev.start(),
                          ev.stop(), 0, E);
    return hipGetLastError();
  }
  hipError_t e = launch_tiles<4>(p, 0, plan.wide, plan, stream);
  if (e == hipSuccess) e = launch_tiles<2>(p, plan.wide, feats, plan, stream);
  if (e != hipSuccess || plan.nsplit == 1) return e;
  const int64_t n = p.T * feats;
  KernelEvents ev(KID_REDUCE);
  hipExtLaunchKernelGGL(k_fp8_sum, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, ev.start(), ev.stop(),
                        0, p.part, plan.nsplit, n, p.C);
  return hipGetLastError();
}

namespace {
// 64 rows and 32 columns j of the source a workgroup; A's transpose goes
// through LDS so that both sides are read and written along their rows.
__global__ __launch_bounds__(256) void k_fp8_pair(const uint16_t* __restrict__ M, int64_t rows, int r, int64_t ldh,
                                                  int transposed, uint16_t* __restrict__ out) {
  __shared__ uint16_t t[64][34];
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int j0 = (int)blockIdx.y * 32;
  const int n = (int)(rows - r0 < 64 ? rows - r0 : 64);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = threadIdx.x + 256 * q;
    const int m = transposed ? e & 63 : e >> 5, j = transposed ? e >> 6 : e & 31;
    uint16_t v = 0;
    if (m < n && j0 + j < r) v = transposed ? M[(int64_t)(j0 + j) * rows + r0 + m] : M[(r0 + m) * r + j0 + j];
    t[m][j] = v;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = threadIdx.x + 256 * q;
    const int m = e >> 5, j = j0 + (e & 31);
    if (m >= n) continue;
    uint16_t* row = out + (r0 + m) * ldh;
    if (j < r) {
      row[j] = t[m][e & 31];
      row[r + j] = t[m][e & 31];
    }
    // the padding behind the pair, shared out among the columns
    for (int64_t c = 2 * r + j; c < ldh; c += 32 * gridDim.y) row[c] = 0;
  }
}
}  // namespace

hipError_t launch_fp8_pair(const uint16_t* M, int64_t rows, int r, int64_t ldh, int transposed, uint16_t* out,
                           hipStream_t stream) {
  KernelEvents ev(KID_FP8_DOWN);
  hipExtLaunchKernelGGL(k_fp8_pair, dim3((unsigned)((rows + 63) / 64), (unsigned)((r + 31) / 32)), dim3(256), 0, stream, ev.start(), ev.stop(), 0,
                        M, rows, r, ldh, transposed, out);
  return hipGetLastError();
}

}  // namespace qlora
