// The adapter's products over the 8-bit form of the layer's input (fp8.hip):
//   down:  U[t][j] = sum_k X[t][k] A[j][k]
//   form:  G[t][j] = sum_n dY[t][n] B[n][j], and the 8-bit form of dY
//   grad:  dA[j][k] = s sum_t G[t][j] X[t][k],  dB[n][j] = s sum_t dY[t][n] U[t][j]
// An e4m3 code times its power-of-two scale is a bf16 value (below 2^128, from
// where on it is an infinity, and down to bf16's subnormal steps of 2^-133, to
// which smaller ones are rounded), so X is restored exactly in registers and
// enters v_mfma_f32_16x16x32_bf16; sums are fp32.  G and U are fp32; for the gradients each is split into three bf16
// terms (hi + mid + lo carry all 24 bits), so the gradients keep fp32
// accuracy, where a pair of terms would round them to about 17 bits.
#include "dma.hpp"
#include "fp8.hpp"
#include "fp8_down.hpp"
#include "fp8_form.hpp"
#include "fp8_sum.hpp"
#include "lds_tr.hpp"
#include "trace.hpp"

namespace qlora {
namespace {

using fp8::absmax_bf16;
using fp8::codes8_bf16;
using fp8::mfma16;
using fp8::restore8;
using fp8::scale_byte;
using fp8::scale_of;
using fp8::u32x4_t;
using ldstr::tr_frag_swz;
using ldstr::tr_swz;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf(const void* p, int64_t bytes) {
  const int32_t n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (int32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, 0x00020000);
}

// ---------------------------------------------------------------------------
// down
//
// A workgroup of eight waves owns 128 tokens and all of U's columns (16 JT) for
// one range of the contraction, a chunk of 128 positions at a time: X's codes
// [128][128 B] and A's rows [16 JT][256 B] are copied straight into one of PD
// LDS stages, PD - 1 chunks ahead; wave w multiplies tokens 16 w .. +15.  The
// range's scales (at most 32 chunks) are in LDS from the start, so nothing but
// the copies is in flight in the loop; as many ranges as fill the CUs, of at most
// 32 chunks (whole dwords of scales), whose sums k_fp8_down_sum adds.  Tiles of 16
// x 16 with fragments loaded from global memory, which cost 64 cache lookups a
// load, took 18 us at 4096 x 8192, r = 64, against 13 here (33.5 MB of codes),
// and 15 to 34 with no second launch at 129 to 500 tokens, against 6 to 13 and
// about 4 for the sums.
// ---------------------------------------------------------------------------
struct DownLaunch {
  Fp8DownParams p;
  int32_t ttiles, nsplit;
  int32_t chunks, chunks_per_split;
};

// Column c < ldh of row t of Us and, for c < r, of U, from the sums v(j).
template <typename SumJ>
__device__ __forceinline__ void down_out(const Fp8DownParams& p, int64_t t, int c, SumJ v_of) {
  uint16_t h = 0;
  if (c < 2 * p.r) {
    const float v = v_of(c < p.r ? c : c - p.r);
    if (p.U && c < p.r) p.U[t * p.r + c] = v;
    uint16_t hi, lo;
    split_bf16(p.s * v, hi, lo);
    h = c < p.r ? hi : lo;
  }
  if (p.Us) p.Us[t * p.ldh + c] = h;
}

__global__ __launch_bounds__(256) void k_fp8_down_sum(DownLaunch L) {
  const Fp8DownParams& p = L.p;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= p.T * p.ldh) return;
  const int64_t t = e / p.ldh;
  down_out(p, t, (int)(e - t * p.ldh), [&](int j) {
    return ordered_sum(L.nsplit, [&](int q) { return p.part[((int64_t)q * p.T + t) * p.r + j]; });
  });
}

constexpr int kDownTok = 128;
constexpr int kDownRange = 32;  // chunks of a range at most

template <int JT>
__global__ __launch_bounds__(512) void k_fp8_down(DownLaunch L) {
  constexpr int PD = JT <= 4 ? 4 : 3;
  constexpr int kX = kDownTok * 128, kA = 16 * JT * 256, kStage = kX + kA;
  constexpr int NA = JT <= 2 ? 1 : JT / 2;  // copies of A a wave and chunk
  constexpr int NC = 2 + NA;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[PD * kStage + 1024];
  __shared__ uint32_t sc[kDownTok][kDownRange / 4];
  const Fp8DownParams& p = L.p;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int i = lane & 15, g = lane >> 4;
  const int split = (int)blockIdx.x / L.ttiles;
  const int64_t t0 = (int64_t)((int)blockIdx.x - split * L.ttiles) * kDownTok;
  const int c_begin = split * L.chunks_per_split;  // a multiple of four
  const int c_end = c_begin + L.chunks_per_split < L.chunks ? c_begin + L.chunks_per_split : L.chunks;
  const int64_t ldx = fp8_scale_ld(p.K);

  for (int e = threadIdx.x; e < kDownTok * (kDownRange / 4); e += 512) {
    const int t = e / (kDownRange / 4), d = e % (kDownRange / 4);
    uint32_t v = 0x7F7F7F7Fu;
    if (t0 + t < p.T && c_begin + 4 * d < c_end) v = reinterpret_cast<const uint32_t*>(p.Xs + (t0 + t) * ldx + c_begin)[d];
    sc[t][d] = v;
  }
  dma::wait_vm<0>();

  const dma::v4i_t rx = dma::rsrc(p.X + t0 * p.K, (p.T - t0) * p.K), ra = dma::rsrc(p.A, (int64_t)p.r * p.K * 2);
  const uint32_t lds0 = LDS_ADDR(lds);
  auto issue = [&](int c) {
    const int ch = c_begin + c;
    const bool in = ch < c_end;
    const uint32_t st = lds0 + (uint32_t)(c % PD * kStage);
    const int64_t k0 = (int64_t)ch * 128;
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // rows 16 w + 8 j .. +7: piece of row R at piece ^ R % 8 ^ R / 8 % 2
      const int R = 16 * wave + 8 * j + (lane >> 3);
      const int64_t k = k0 + 16 * ((lane & 7) ^ (lane >> 3) ^ j);
      dma::copy16(rx, in && t0 + R < p.T && k < p.K ? (uint32_t)(R * p.K + k) : dma::kOob, st + 2048 * wave + 1024 * j);
    }
#pragma unroll
    for (int j = 0; j < NA; ++j) {  // four rows of A: piece of row R at piece ^ R % 16
      const int blk = NA * wave + j;
      const int R = 4 * blk + (lane >> 4);
      const int64_t k = k0 + 8 * (i ^ (R & 15));
      // with 16 columns the last waves have nothing to copy: so that every wave
      // counts alike, theirs read nothing and fill the kilobyte behind the stages
      const bool mine = blk < 4 * JT;
      dma::copy16(ra, in && mine && R < p.r && k < p.K ? (uint32_t)((R * p.K + k) * 2) : dma::kOob,
                  mine ? st + kX + 1024 * blk : lds0 + PD * kStage);
    }
  };

  f32x4_t acc[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) acc[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int n = c_end - c_begin;
#pragma unroll
  for (int c = 0; c < PD - 1; ++c) issue(c);
  for (int c = 0; c < n; ++c) {
    dma::wait_vm<(PD - 2) * NC>();  // this wave's copies of chunk c have landed
    lds_barrier();                  // everybody's have, and chunk c - 1 is read
    issue(c + PD - 1);
    const uint8_t* X = lds + c % PD * kStage;
    const uint8_t* A = X + kX;
    const int R = 16 * wave + i, sw = (i & 7) ^ (i >> 3);
    const u32x4_t x0 = *reinterpret_cast<const u32x4_t*>(X + R * 128 + (((2 * g) ^ sw) << 4));
    const u32x4_t x1 = *reinterpret_cast<const u32x4_t*>(X + R * 128 + (((2 * g + 1) ^ sw) << 4));
    const float k = scale_of(sc[R][c >> 2] >> (8 * (c & 3)) & 0xFFu);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4_t x = q < 2 ? x0 : x1;
      const bf16x8_t xa = __builtin_bit_cast(bf16x8_t, restore8(x[2 * (q & 1)], x[2 * (q & 1) + 1], k));
#pragma unroll
      for (int jt = 0; jt < JT; ++jt)
        acc[jt] = mfma16(xa, *reinterpret_cast<const bf16x8_t*>(A + (16 * jt + i) * 256 + (((4 * g + q) ^ i) << 4)), acc[jt]);
    }
  }
  dma::wait_vm<0>();  // no copy may land in LDS that is no longer this workgroup's

  // lane l, value v: token 16 w + 4 (l/16) + v, column 16 jt + l % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t t = t0 + 16 * wave + 4 * g + v;
    if (t >= p.T) continue;
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int j = 16 * jt + i;
      if (j < p.r) p.part[((int64_t)split * p.T + t) * p.r + j] = acc[jt][v];
    }
  }
}

int down_ranges(int64_t T, int64_t K, int32_t& per) {
  const int64_t tiles = (T + kDownTok - 1) / kDownTok, chunks = (K + 127) / 128;
  int64_t s = 256 / tiles;
  if (s < (chunks + kDownRange - 1) / kDownRange) s = (chunks + kDownRange - 1) / kDownRange;
  per = (int32_t)(((chunks + s - 1) / s + 3) / 4 * 4);
  return (int)((chunks + per - 1) / per);
}

// ---------------------------------------------------------------------------
// form: G and the 8-bit form of dY in one pass over it
//
// As down: a workgroup of eight waves owns 128 tokens for one
// range of the contraction, a chunk of 128 columns at a time, dY's [128][256 B]
// and B's [128][32 JT B] copied into LDS two chunks ahead.  A lane holds 32
// columns of one row, its share of four MFMAs; four lanes have the row's block
// and find its largest value, and the lane writes its codes.  B's contraction
// runs down its rows: transposing reads.
//
// Bound by HBM's latency: 4096 x 8192, r = 64 (101 MB read and written): 24 us,
// 4.2 TB/s, against 16 + 16 for G and the form in launches of their own, which
// read dY twice; a whole backward takes 1 to 10% less, from 4 tokens (27.7 us
// against 30.8, 4096 x 4096, r = 16) to 4096 (291 against 296).  Vector
// work (the largest value and the codes on 16 bits instead of 32) and the order
// of the chunks (other ranges' tiles starting at other columns) changed nothing.
// ---------------------------------------------------------------------------
struct FormLaunch {
  Fp8FormParams p;
  int32_t ttiles, chunks, chunks_per_split;
};

template <int JT>
__global__ __launch_bounds__(512) void k_fp8_form(FormLaunch L) {
  constexpr int PD = 3;
  constexpr int QLD = 16 * JT, PPR = 2 * JT;  // a row of B: elements, 16-byte pieces
  constexpr int kP = kDownTok * 256, kB = 128 * QLD * 2, kStage = kP + kB;
  constexpr int NB = JT <= 2 ? 1 : JT / 2;  // copies of B a wave and chunk
  constexpr int NC = 4 + NB;
  constexpr int NS = 4;                     // stores a wave and chunk
  __shared__ __attribute__((aligned(1024))) uint8_t lds[PD * kStage + 1024];
  __shared__ uint32_t sc[kDownTok][kDownRange / 4];
  const Fp8FormParams& p = L.p;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int i = lane & 15, g = lane >> 4;
  const int split = __builtin_amdgcn_readfirstlane((int)blockIdx.x / L.ttiles);
  const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane((int)blockIdx.x - split * L.ttiles) * kDownTok;
  const int c_begin = split * L.chunks_per_split;  // a multiple of four
  const int c_end = c_begin + L.chunks_per_split < L.chunks ? c_begin + L.chunks_per_split : L.chunks;
  const int n = c_end - c_begin;

  const dma::v4i_t rp = dma::rsrc(p.dY + t0 * p.N, (p.T - t0) * p.N * 2), rb = dma::rsrc(p.B, p.N * p.r * 2);
  // (without codes an empty range, which drops the stores)
  const __amdgpu_buffer_rsrc_t rc = buf(p.codes + t0 * p.N, p.codes ? (p.T - t0) * p.N : 0);
  const uint32_t lds0 = LDS_ADDR(lds);
  auto issue = [&](int c) {
    const bool in = c < n;
    const uint32_t st = lds0 + (uint32_t)(c % PD * kStage);
    const int64_t n0 = (int64_t)(c_begin + c) * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // rows 16 w + 4 j .. +3: piece of row R at piece ^ R % 16
      const int R = 16 * wave + 4 * j + (lane >> 4);
      const int64_t col = n0 + 8 * (i ^ (R & 15));
      dma::copy16(rp, in && t0 + R < p.T && col < p.N ? (uint32_t)((R * p.N + col) * 2) : dma::kOob,
                  st + 4096 * wave + 1024 * j);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int blk = NB * wave + j;
      const int R = blk * (64 / PPR) + lane / PPR;
      const int col = 8 * ((lane & (PPR - 1)) ^ tr_swz(R, PPR));
      // with 16 columns the last waves have nothing to copy, as above
      const bool mine = blk < 4 * JT;
      dma::copy16(rb, in && mine && n0 + R < p.N && col < p.r ? (uint32_t)(((n0 + R) * p.r + col) * 2) : dma::kOob,
                  mine ? st + kP + 1024 * blk : lds0 + PD * kStage);
    }
  };

  for (int e = threadIdx.x; e < kDownTok * (kDownRange / 4); e += 512) (&sc[0][0])[e] = 0x7F7F7F7Fu;
  f32x4_t acc[JT];
#pragma unroll
  for (int jt = 0; jt < JT; ++jt) acc[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < PD - 1; ++c) issue(c);
  const int R = 16 * wave + i;
  for (int c = 0; c < n; ++c) {
    // this wave's copies of chunk c have landed; behind them went out those of
    // the next PD - 2 chunks and, from the third chunk on, two chunks' stores
    if (c >= PD - 1) dma::wait_vm<(PD - 2) * NC + (PD - 1) * NS>();
    else dma::wait_vm<(PD - 2) * NC>();
    lds_barrier();  // everybody's have, and chunk c - 1 is read
    issue(c + PD - 1);
    const uint8_t* P = lds + c % PD * kStage;
    const uint16_t* B = reinterpret_cast<const uint16_t*>(P + kP);
    u32x4_t x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<const u32x4_t*>(P + R * 256 + (((4 * q + g) ^ i) << 4));
    uint32_t m = absmax_bf16(16, [&](int q) -> uint32_t { return x[q >> 2][q & 3]; });
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bf16x8_t xa = __builtin_bit_cast(bf16x8_t, x[q]);
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) acc[jt] = mfma16(xa, tr_frag_swz(B, QLD, 32 * q + 8 * g, 16 * jt), acc[jt]);
    }
    const uint32_t m16 = (uint32_t)__shfl_xor((int)m, 16);
    m = m16 > m ? m16 : m;
    const uint32_t m32 = (uint32_t)__shfl_xor((int)m, 32);
    m = m32 > m ? m32 : m;
    const uint32_t e = scale_byte(m);
    if (g == 0) reinterpret_cast<uint8_t*>(sc[R])[c] = (uint8_t)e;
    const int64_t n0 = (int64_t)(c_begin + c) * 128 + 8 * g;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t col = n0 + 32 * q;
      __builtin_amdgcn_raw_buffer_store_b64(codes8_bf16(x[q][0], x[q][1], x[q][2], x[q][3], e), rc,
                                            t0 + R < p.T && col < p.N ? (uint32_t)(R * p.N + col) : dma::kOob, 0, 0);
    }
  }
  dma::wait_vm<0>();  // no copy may land in LDS that is no longer this workgroup's
  lds_barrier();

  // whole dwords of scales, the row's padding in the last
  const int64_t lds_ = fp8_scale_ld(p.N);
  for (int e = threadIdx.x; e < kDownTok * (kDownRange / 4); e += 512) {
    const int t = e / (kDownRange / 4), d = e % (kDownRange / 4);
    if (p.codes && t0 + t < p.T && 4 * d < n) reinterpret_cast<uint32_t*>(p.scales + (t0 + t) * lds_ + c_begin)[d] = sc[t][d];
  }
  // lane l, value v: token 16 w + 4 (l/16) + v, column 16 jt + l % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t t = t0 + 16 * wave + 4 * g + v;
    if (t >= p.T) continue;
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int j = 16 * jt + i;
      if (j < p.r) p.part[((int64_t)split * p.T + t) * p.r + j] = acc[jt][v];
    }
  }
}

// ---------------------------------------------------------------------------
// grad: out[m][j] = s sum_t P[t][m] Q[t][j]
//
// A workgroup of eight waves owns 256 columns m of P (wave w: 32 of them) and
// every j for one range of tokens, in chunks of 32 tokens: P's tile goes
// through registers (restored, if it is codes) into LDS as bf16 [32][256], Q's
// as three planes of bf16 [32][16 JT].  Both operands are read back with
// transposing reads, the contraction running down the rows.
//
// What bounds it is LDS: a wave reads 2 + 3 JT fragments of 1 KB for 6 JT
// MFMAs, and Q's three planes are the same for all eight waves.  4096 tokens,
// 8192 x 8192, r = 64 (101 MB, 19 us at a copy's rate): 38 us; with four waves,
// 64 columns a wave: 45; with 512 columns: 56 (fewer workgroups a CU).
// ---------------------------------------------------------------------------
constexpr int kGradM = 256;
constexpr int kGradChunk = 32;

struct GradLaunch {
  Fp8GradParams p;
  int32_t slabs_a, slabs_b;  // of dA's columns (K) and of dB's rows (N)
  int32_t nsplit, chunks, chunks_per_split;
};

// second: dB, over bf16 rows; else dA, over codes.
template <int JT, bool second>
__device__ __forceinline__ void grad_body(const GradLaunch& L, int slab, int split,
                                          uint16_t (*lds)[kGradChunk * (kGradM + 48 * JT)]) {
  constexpr int QLD = 16 * JT;
  constexpr int kP = kGradChunk * kGradM, kQ = kGradChunk * QLD;  // elements
  const Fp8GradParams& p = L.p;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int i = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)slab * kGradM;
  const int64_t D = second ? p.N : p.K;
  const float* Q = second ? p.U : p.G;
  const int r = p.r;
  const int64_t ldx = fp8_scale_ld(p.K);
  const int c_begin = split * L.chunks_per_split;
  const int c_end = c_begin + L.chunks_per_split < L.chunks ? c_begin + L.chunks_per_split : L.chunks;

  // thread: row tid / 16 of the chunk, 16 columns of P and JT of Q
  const int row = threadIdx.x >> 4, pc = threadIdx.x & 15;
  const int64_t col = m0 + 16 * pc;
  struct Chunk {
    u32x4_t p[second ? 2 : 1];
    uint32_t s;
    float q[JT];
  };
  // (buffer loads: what lies outside reads zero, with nothing to wait for)
  const __amdgpu_buffer_rsrc_t rp = second ? buf(p.dY, p.T * p.N * 2) : buf(p.X, p.T * p.K);
  const __amdgpu_buffer_rsrc_t rs = buf(p.Xs, second ? 0 : p.T * ldx), rq = buf(Q, p.T * r * 4);
  auto fetch = [&](Chunk& c, int ch) {
    const uint32_t t = (uint32_t)ch * kGradChunk + row;
    const bool in = ch < c_end && t < p.T, ok = in && col < D;
    const uint32_t at = (uint32_t)((t * D + col) * (second ? 2 : 1));
    c.p[0] = __builtin_amdgcn_raw_buffer_load_b128(rp, ok ? at : dma::kOob, 0, 0);
    if (second) c.p[second ? 1 : 0] = __builtin_amdgcn_raw_buffer_load_b128(rp, ok ? at + 16 : dma::kOob, 0, 0);
    else c.s = __builtin_amdgcn_raw_buffer_load_b8(rs, ok ? (uint32_t)(t * ldx + (col >> 7)) : dma::kOob, 0, 0);
#pragma unroll
    for (int q = 0; q < JT; ++q) {
      const int j = pc + 16 * q;
      c.q[q] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(rq, in && j < r ? (t * (uint32_t)r + j) * 4u : dma::kOob, 0, 0));
    }
  };
  auto stage = [&](const Chunk& c, int buf) {
    uint16_t* P = lds[buf];
    u32x4_t a = c.p[0], b = c.p[second ? 1 : 0];
    if (!second) {
      const float k = scale_of(c.s);
      b = restore8(c.p[0][2], c.p[0][3], k);
      a = restore8(c.p[0][0], c.p[0][1], k);
    }
    const int s = tr_swz(row, kGradM / 8);
    *reinterpret_cast<u32x4_t*>(P + row * kGradM + (((2 * pc) ^ s) << 3)) = a;
    *reinterpret_cast<u32x4_t*>(P + row * kGradM + (((2 * pc + 1) ^ s) << 3)) = b;
    const int sq = tr_swz(row, QLD / 8);
#pragma unroll
    for (int q = 0; q < JT; ++q) {
      const int j = pc + 16 * q;
      const float v = p.s * c.q[q];
      uint16_t h, m, l;
      split_bf16(v, h, m);
      const float rest = v - bf16_bits_to_f32(h);
      l = f32_to_bf16_bits(rest - bf16_bits_to_f32(m));
      uint16_t* dst = P + kP + row * QLD + ((((j >> 3) ^ sq) << 3) | (j & 7));
      dst[0] = h;
      dst[kQ] = m;
      dst[2 * kQ] = l;
    }
  };

  f32x4_t acc[2][JT];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) acc[a][jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  Chunk c0, c1;
  auto body = [&](Chunk& c, int ch, int buf) {
    stage(c, buf);
    fetch(c, ch + 2);
    lds_barrier();  // the chunk is staged; every wave is done with the other buffer
    const uint16_t* P = lds[buf];
    bf16x8_t pa[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) pa[a] = tr_frag_swz(P, kGradM, 8 * g, 32 * wave + 16 * a);
#pragma unroll
    for (int jt = 0; jt < JT; ++jt)
#pragma unroll
      for (int q = 2; q >= 0; --q) {  // the smallest terms first
        const bf16x8_t qb = tr_frag_swz(P + kP + q * kQ, QLD, 8 * g, 16 * jt);
#pragma unroll
        for (int a = 0; a < 2; ++a) acc[a][jt] = mfma16(pa[a], qb, acc[a][jt]);
      }
  };
  fetch(c0, c_begin);
  fetch(c1, c_begin + 1);
  for (int ch = c_begin; ch < c_end; ch += 2) {
    body(c0, ch, 0);
    if (ch + 1 < c_end) body(c1, ch + 1, 1);
  }

  // lane l, value v: column m = 32 wave + 16 a + 4 (l/16) + v, j = 16 jt + l % 16
  const bool split_out = L.nsplit > 1;
  float* out = second ? p.dB : p.dA;
  if (split_out) out = p.part + (int64_t)split * r * (p.K + p.N) + (second ? (int64_t)r * p.K : 0);
  const bool add = !split_out && p.accumulate;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int64_t m = m0 + 32 * wave + 16 * a + 4 * g;
    if (m >= D) continue;
#pragma unroll
    for (int jt = 0; jt < JT; ++jt) {
      const int j = 16 * jt + i;
      if (j >= r) continue;
      if (second) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float* dst = out + (m + v) * r + j;
          *dst = add ? *dst + acc[a][jt][v] : acc[a][jt][v];
        }
      } else {
        f32x4_t* dst = reinterpret_cast<f32x4_t*>(out + (int64_t)j * D + m);
        f32x4_t o = acc[a][jt];
        if (add) {
          const f32x4_t w = *dst;
#pragma unroll
          for (int v = 0; v < 4; ++v) o[v] = w[v] + o[v];
        }
        *dst = o;
      }
    }
  }
}

template <int JT>
__global__ __launch_bounds__(512, JT <= 4 ? 4 : 2) void k_fp8_grad(GradLaunch L) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[2][kGradChunk * (kGradM + 48 * JT)];
  const int slabs = L.slabs_a + L.slabs_b;
  const int split = (int)blockIdx.x / slabs, slab = (int)blockIdx.x - split * slabs;
  if (slab >= L.slabs_a) grad_body<JT, true>(L, slab - L.slabs_a, split, lds);
  else grad_body<JT, false>(L, slab, split, lds);
}

// The token ranges' partial sums in order (dA's, then dB's), four elements a
// thread; K and N are multiples of 64, so no piece straddles the two.
__global__ __launch_bounds__(256) void k_fp8_grad_sum(GradLaunch L) {
  const Fp8GradParams& p = L.p;
  const int64_t na = (int64_t)p.r * p.K, n = na + (int64_t)p.r * p.N;
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= n) return;
  f32x4_t v = ordered_sum(L.nsplit, [&](int q) { return *reinterpret_cast<const f32x4_t*>(p.part + q * n + e); });
  f32x4_t* dst = reinterpret_cast<f32x4_t*>(e < na ? p.dA + e : p.dB + (e - na));
  if (p.accumulate) {
    const f32x4_t o = *dst;
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = o[x] + v[x];
  }
  *dst = v;
}

// Token ranges: 512 workgroups in all, of four chunks each at least.  r = 64, G
// and its sum included: 8192 x 8192, 4096 tokens: 63 us, as with 256 workgroups,
// with 1024 79; 22016 x 8192: 121 against 132 and 131 (1333 tokens: 57.5, 55 and
// 66).  At most 16 ranges; with 8 or 32 the times are the same within a few
// percent.
int grad_splits(int64_t T, int64_t K, int64_t N) {
  const int64_t slabs = (K + kGradM - 1) / kGradM + (N + kGradM - 1) / kGradM;
  const int64_t chunks = (T + kGradChunk - 1) / kGradChunk;
  int64_t s = 512 / slabs;
  if (s > chunks / 4) s = chunks / 4;
  if (s > 16) s = 16;
  return (int)(s < 1 ? 1 : s);
}

}  // namespace

size_t fp8_down_part_bytes(int64_t T, int64_t K, int r) {
  int32_t per;
  return (size_t)down_ranges(T, K, per) * T * r * 4;
}

hipError_t launch_fp8_down(const Fp8DownParams& p, hipStream_t stream) {
  if (!p.part || p.part_bytes < fp8_down_part_bytes(p.T, p.K, p.r)) return hipErrorInvalidValue;
  DownLaunch L{};
  L.p = p;
  L.chunks = (int32_t)((p.K + 127) / 128);
  L.nsplit = down_ranges(p.T, p.K, L.chunks_per_split);
  L.ttiles = (int32_t)((p.T + kDownTok - 1) / kDownTok);
  {
    KernelEvents ev(KID_FP8_DOWN);
    const hipEvent_t e0 = ev.start(), e1 = ev.stop();
    const dim3 grid((unsigned)(L.ttiles * L.nsplit)), block(512);
    const int jt = (p.r + 15) / 16;
    if (jt == 1) hipExtLaunchKernelGGL(k_fp8_down<1>, grid, block, 0, stream, e0, e1, 0, L);
    else if (jt == 2) hipExtLaunchKernelGGL(k_fp8_down<2>, grid, block, 0, stream, e0, e1, 0, L);
    else if (jt <= 4) hipExtLaunchKernelGGL(k_fp8_down<4>, grid, block, 0, stream, e0, e1, 0, L);
    else hipExtLaunchKernelGGL(k_fp8_down<8>, grid, block, 0, stream, e0, e1, 0, L);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  KernelEvents ev(KID_REDUCE);
  hipExtLaunchKernelGGL(k_fp8_down_sum, dim3((unsigned)((p.T * p.ldh + 255) / 256)), dim3(256), 0, stream, ev.start(),
                        ev.stop(), 0, L);
  return hipGetLastError();
}

bool fp8_form_ok(int r) { return r > 0 && r <= 64 && r % 8 == 0; }

size_t fp8_form_part_bytes(int64_t T, int64_t N, int r) {
  int32_t per;
  return (size_t)down_ranges(T, N, per) * T * r * 4;
}

hipError_t launch_fp8_form(const Fp8FormParams& p, hipStream_t stream) {
  if (!fp8_form_ok(p.r) || !p.part || p.part_bytes < fp8_form_part_bytes(p.T, p.N, p.r)) return hipErrorInvalidValue;
  FormLaunch L{};
  L.p = p;
  L.chunks = (int32_t)((p.N + 127) / 128);
  DownLaunch S{};
  S.nsplit = down_ranges(p.T, p.N, L.chunks_per_split);
  S.p.T = p.T; S.p.r = p.r; S.p.s = p.s; S.p.U = p.G; S.p.Us = p.Gs; S.p.ldh = p.ldh; S.p.part = p.part;
  L.ttiles = (int32_t)((p.T + kDownTok - 1) / kDownTok);
  {
    KernelEvents ev(KID_LORA_G);
    const hipEvent_t e0 = ev.start(), e1 = ev.stop();
    const dim3 grid((unsigned)(L.ttiles * S.nsplit)), block(512);
    const int jt = (p.r + 15) / 16;
    if (jt == 1) hipExtLaunchKernelGGL(k_fp8_form<1>, grid, block, 0, stream, e0, e1, 0, L);
    else if (jt == 2) hipExtLaunchKernelGGL(k_fp8_form<2>, grid, block, 0, stream, e0, e1, 0, L);
    else hipExtLaunchKernelGGL(k_fp8_form<4>, grid, block, 0, stream, e0, e1, 0, L);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  KernelEvents ev(KID_REDUCE);
  hipExtLaunchKernelGGL(k_fp8_down_sum, dim3((unsigned)((p.T * p.ldh + 255) / 256)), dim3(256), 0, stream, ev.start(),
                        ev.stop(), 0, S);
  return hipGetLastError();
}

size_t fp8_grad_part_bytes(int64_t T, int64_t K, int64_t N, int r) {
  const int s = grad_splits(T, K, N);
  return s > 1 ? (size_t)s * r * (K + N) * 4 : 0;
}

hipError_t launch_fp8_grad(const Fp8GradParams& p, hipStream_t stream) {
  GradLaunch L{};
  L.p = p;
  L.slabs_a = (int32_t)((p.K + kGradM - 1) / kGradM);
  L.slabs_b = (int32_t)((p.N + kGradM - 1) / kGradM);
  L.chunks = (int32_t)((p.T + kGradChunk - 1) / kGradChunk);
  L.nsplit = grad_splits(p.T, p.K, p.N);
  L.chunks_per_split = (L.chunks + L.nsplit - 1) / L.nsplit;
  if (L.nsplit > 1 && (!p.part || p.part_bytes < fp8_grad_part_bytes(p.T, p.K, p.N, p.r))) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((L.slabs_a + L.slabs_b) * L.nsplit)), block(512);
  const int jt = (p.r + 15) / 16;
  {
    KernelEvents ev(KID_FP8_GRAD);
    const hipEvent_t e0 = ev.start(), e1 = ev.stop();
    if (jt == 1) hipExtLaunchKernelGGL(k_fp8_grad<1>, grid, block, 0, stream, e0, e1, 0, L);
    else if (jt == 2) hipExtLaunchKernelGGL(k_fp8_grad<2>, grid, block, 0, stream, e0, e1, 0, L);
    else if (jt <= 4) hipExtLaunchKernelGGL(k_fp8_grad<4>, grid, block, 0, stream, e0, e1, 0, L);
    else hipExtLaunchKernelGGL(k_fp8_grad<8>, grid, block, 0, stream, e0, e1, 0, L);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || L.nsplit == 1) return e;
  const int64_t n = (int64_t)p.r * (p.K + p.N);
  KernelEvents ev(KID_REDUCE);
  hipExtLaunchKernelGGL(k_fp8_grad_sum, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, ev.start(),
                        ev.stop(), 0, L);
  return hipGetLastError();
}

}  // namespace qlora
