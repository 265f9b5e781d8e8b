// Products of two 8-bit forms on 256 x 256 output tiles (see fp8_gemm.hip for
// the products and for what the matrix instruction does).
//
// One workgroup of four waves per CU, one wave per SIMD with 512 registers.
// Wave (a, b) owns features 128 a .. +127 and tokens 128 b .. +127: 4 x 4
// tiles of 32 x 32, 256 fp32 accumulators a lane.
// v_mfma_scale_f32_32x32x64_f8f6f4 takes half a block of 128: lane l holds row
// (column) l % 32 and 32 consecutive codes, those from 32 (l / 32) of the 64.
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

constexpr int WT = 256, WF = 256;
constexpr uint32_t kSlot = 256 * 128;
constexpr uint32_t kSlots = 5;
constexpr int kOutLd = WF + 8;
constexpr int kLds = kSlots * kSlot;
static_assert(WT * kOutLd * 2 <= kLds, "the output tile fits over the slots");

// the n-th slot after the one at byte o
__device__ __forceinline__ uint32_t slot_after(uint32_t o, uint32_t n) {
  return o + n * kSlot < kLds ? o + n * kSlot : o + n * kSlot - kLds;
}

struct WideLaunch {
  Fp8Params p;
  int32_t mt, nt, group;  // token tiles, feature tiles, token tiles walked together
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf(const void* p, int64_t bytes) {
  const int32_t n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (int32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, n, 0x00020000);
}

template <int Q>
__device__ __forceinline__ f32x16_t mfma8(v8i_t a, v8i_t b, f32x16_t c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, Q, (int)sa, Q, (int)sb);
}

// A copy into LDS that the compiler does not count (see dma.hpp): behind one
// that it knows of, it would wait for every copy in flight before a
// transposing read.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_uncounted(dma::v4i_t r, uint32_t voff, uint32_t soff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(dst), "v"(voff), "s"(r), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

struct Frags {
  u32x4_t x[4][2], w[4][2];
};

template <bool DX>
__global__ __launch_bounds__(256, 1) void k_fp8_wide(WideLaunch L) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const Fp8Params& p = L.p;
  // runs of consecutive tiles go to one XCD; in their order, groups of token
  // tiles are walked feature tile by feature tile
  const uint32_t mt = (uint32_t)L.mt, nt = (uint32_t)L.nt, gm = (uint32_t)L.group;
  const uint32_t run = (mt * nt + 7) / 8;
  const uint32_t order = blockIdx.x % 8 * run + blockIdx.x / 8;
  if (order >= mt * nt) return;
  const uint32_t first = order / (gm * nt) * gm;
  const uint32_t rows = mt - first < gm ? mt - first : gm;
  const uint32_t in_group = order - first * nt;
  // (in scalar registers: they go into the buffer resources)
  const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane((first + in_group % rows) * WT);
  const int64_t f0 = (int64_t)__builtin_amdgcn_readfirstlane(in_group / rows * WF);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wf = 128 * (wave & 1), wt = 128 * (wave >> 1);
  const int g = lane >> 5, c32 = lane & 31, i16 = lane & 15;
  const int64_t len = DX ? p.Nw : p.Kw, feats = DX ? p.Kw : p.Nw;
  const uint32_t nsteps = __builtin_amdgcn_readfirstlane((uint32_t)(len / 64));

  const __amdgpu_buffer_rsrc_t rx = buf(p.X + t0 * len, (p.T - t0) * len);
  const __amdgpu_buffer_rsrc_t rw = DX ? buf(p.W + f0, p.Nw * p.Kw - f0) : buf(p.W + f0 * len, (feats - f0) * len);
  const dma::v4i_t ax = dma::rsrc(p.X + t0 * len, (p.T - t0) * len), aw = dma::rsrc(p.W + f0, p.Nw * p.Kw - f0);  // dx
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(LDS_ADDR(lds));
  const __amdgpu_buffer_rsrc_t rs = buf(p.Xs, p.T * fp8_scale_ld(len));

  // copies of a pair of steps: eight kilobytes of each operand a wave.  Rows
  // past the last token or feature read zeros.
  uint32_t xoff[8], woff[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int R = 64 * wave + 8 * j + (lane >> 3);
    const int chunk = (lane & 7) ^ (lane >> 3) ^ (j & 1);
    xoff[j] = t0 + R < p.T ? (uint32_t)(R * len + chunk * 16) : dma::kOob;
    if (DX) {
      const int n = 32 * wave + 4 * j + (lane >> 4);
      const int piece = i16 ^ (2 * (n & 7));
      woff[j] = f0 + piece * 16 < feats ? (uint32_t)(n * p.Kw + piece * 16) : dma::kOob;
    } else {
      woff[j] = f0 + R < feats ? (uint32_t)(R * len + chunk * 16) : dma::kOob;
    }
  }
  const uint32_t wpair = DX ? (uint32_t)(128 * p.Kw) : 128u;
  const uint32_t pairs = (nsteps + 1) / 2;
  // copy j (0 .. 7) of X's or W's pair `pr` into a slot
  auto copy_x = [&](uint32_t pr, uint32_t slot, int j) {
    const uint32_t at = pr < pairs ? pr : pairs - 1;
    if (DX) copy16_uncounted(ax, xoff[j], at * 128u, lds0 + slot + 8192 * wave + 1024 * j);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(lds + slot + 8192 * wave + 1024 * j), 16, xoff[j], at * 128u, 0, 0);
  };
  auto copy_w = [&](uint32_t pr, uint32_t slot, int j) {
    const uint32_t at = pr < pairs ? pr : pairs - 1;
    if (DX) copy16_uncounted(aw, woff[j], at * wpair, lds0 + slot + 8192 * wave + 1024 * j);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(lds + slot + 8192 * wave + 1024 * j), 16, woff[j], at * wpair, 0, 0);
  };

  // scales: a dword holds the bytes of four blocks, eight steps
  const uint32_t groups = (nsteps + 7) / 8;
  uint32_t soff[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t row = t0 + wt + 32 * t + c32;
    soff[t] = (uint32_t)((row < p.T ? row : p.T - 1) * fp8_scale_ld(len));
  }
  // X's: a dword a group; for dx, whose copies are uncounted and drained by
  // the wait for a counted load, four dwords in every fourth group (3% faster
  // there, and as much slower where the copies are counted)
  auto load_sx = [&](uint32_t gr, int t) {
    return __builtin_amdgcn_raw_buffer_load_b32(rs, soff[t], (gr < groups ? gr : groups - 1) * 4u, 0);
  };
  auto load_sx4 = [&](uint32_t quad, int t) { return __builtin_amdgcn_raw_buffer_load_b128(rs, soff[t], quad * 16u, 0); };
  // the wave's 128 features are one block of the weight: its bytes lie in one
  // row of the weight's scales, or, for dx, in one column of them
  const int64_t fb = __builtin_amdgcn_readfirstlane((uint32_t)((f0 + wf < feats ? f0 + wf : f0) / 128));
  const int64_t ldw = fp8_scale_ld(p.Kw);
  struct SwRaw {
    uint32_t v[4];
  };
  auto load_sw = [&](uint32_t gr) {
    const uint32_t at = gr < groups ? gr : groups - 1;
    SwRaw r{};
    if (!DX) {
      r.v[0] = *(const_u32)(p.Ws + fb * ldw + 4 * at);
    } else {
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q)
        r.v[q] = *(const_u32)(p.Ws + (4 * at + q < pairs ? 4 * at + q : pairs - 1) * ldw + (fb & ~3LL));
    }
    return r;
  };
  auto sw_of = [&](const SwRaw& r) -> uint32_t {
    if (!DX) return r.v[0];
    const uint32_t sh = 8 * (uint32_t)(fb & 3);
    return (r.v[0] >> sh & 0xFFu) | (r.v[1] >> sh & 0xFFu) << 8 | (r.v[2] >> sh & 0xFFu) << 16 | (r.v[3] >> sh) << 24;
  };

  // fragment reads of half h of a pair; tile t's are 4096 bytes on (dx: rows
  // 64 h + 8 q are 256 (64 h + 8 q) bytes on)
  const int sw = (c32 & 7) ^ ((c32 >> 3) & 1);
  uint32_t xpos[2][2], wpos[4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 2; ++e) xpos[h][e] = (uint32_t)(c32 * 128 + (((4 * h + 2 * g + e) ^ sw) << 4));
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int piece = (wf >> 4) + 2 * f + ((lane >> 4) & 1);
    wpos[f] = (uint32_t)((32 * g + (i16 >> 1)) * 256 + ((piece ^ (i16 & 14)) << 4) + 8 * (i16 & 1));
  }
  auto read_x = [&](Frags& F, uint32_t slot, int h, int t, int e) {
    F.x[t][e] = *reinterpret_cast<const u32x4_t*>(lds + (slot + wt * 128) + xpos[h][e] + 4096 * t);
  };
  auto read_w = [&](Frags& F, uint32_t slot, int h, int f, int e) {
    if (DX) {
#pragma unroll
      for (int q = 2 * e; q < 2 * e + 2; ++q) {
        const v2i_t v = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i_t*)((lds_u8_t*)lds + slot + wpos[f] + 256 * (64 * h + 8 * q)));
        F.w[f][e][2 * (q & 1)] = (uint32_t)v[0];
        F.w[f][e][2 * (q & 1) + 1] = (uint32_t)v[1];
      }
    } else {
      F.w[f][e] = *reinterpret_cast<const u32x4_t*>(lds + (slot + wf * 128) + xpos[h][e] + 4096 * f);
    }
  };
  // read n (0 .. 15) of a step's fragments, in the order the MFMAs need them
  auto read = [&](Frags& F, uint32_t xslot, uint32_t wslot, int h, int n) {
    if (n < 2) read_w(F, wslot, h, 0, n);
    else if (n < 10) read_x(F, xslot, h, (n - 2) >> 1, n & 1);
    else read_w(F, wslot, h, 1 + ((n - 10) >> 1), n & 1);
  };

  f32x16_t acc[4][4];  // [feature tile][token tile]
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[f][t][v] = 0.0f;

  uint32_t sx[4], sxn[4], swc;
  u32x4_t sxq[4];
  SwRaw swn;
  Frags F[2];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (DX) {
      sxq[t] = load_sx4(0, t);
      sx[t] = sxq[t][0];
    } else {
      sx[t] = sxn[t] = load_sx(0, t);
    }
  }
  swn = load_sw(0);
  swc = sw_of(swn);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) copy_x(c, 2 * c * kSlot, j);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 8; ++j) copy_w(c, (2 * c + 1) * kSlot, j);
    __builtin_amdgcn_sched_barrier(0);
  }
  dma::wait_vm<16>();  // the first pair's copies have landed; the second's went out after them
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int n = 0; n < 16; ++n) read(F[0], 0, kSlot, 0, n);

  uint32_t slot = 0;  // X of the step's pair; W's is the next one
  auto step = [&](uint32_t u, auto j_) {
    constexpr int J = decltype(j_)::value, Q = J / 2;
    constexpr bool odd = J % 2 != 0;
    Frags& C = F[odd];
    Frags& Nx = F[!odd];
    const uint32_t pr = u / 2;
    // the next step's fragments: the pair's second half, or the next pair's first
    const uint32_t rx_ = odd ? slot_after(slot, 2) : slot, rw_ = odd ? slot_after(slot, 3) : slot_after(slot, 1);
    const uint32_t fill = odd ? slot : slot_after(slot, 4);
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const int f = m >> 2, t = m & 3;
      const u32x4_t w0 = C.w[f][0], w1 = C.w[f][1], x0 = C.x[t][0], x1 = C.x[t][1];
      acc[f][t] = mfma8<Q>(v8i_t{(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]},
                           v8i_t{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]},
                           acc[f][t], swc, sx[t]);
      if (odd) {
        if (m == 1) {
          // the next pair's copies have landed (after them went out the eight
          // of X in the step before, and the scales' four if that was J = 2),
          // and this wave's fragments of the pair are read
          dma::wait_vm<!DX && J == 3 ? 12 : 8>();
          lds_barrier();
        }
        if (m >= 2) read(Nx, rx_, rw_, 0, m - 2);
        if (m >= 14) read(Nx, rx_, rw_, 0, m);
        if (m >= 2 && m % 2 == 0) copy_w(pr + 2, fill, m / 2 - 1);
        if (m == 15) copy_w(pr + 2, fill, 7);
      } else {
        read(Nx, rx_, rw_, 1, m);
        if (m % 2 == 0) copy_x(pr + 2, fill, m / 2);
        if (!DX && J == 2 && m % 4 == 1) sxn[m / 4] = load_sx(u / 8 + 1, m / 4);
        if (J == 2 && m == 8) swn = load_sw(u / 8 + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (odd) slot = slot_after(slot, 2);
  };
  auto steps8 = [&](uint32_t u) {
    step(u, std::integral_constant<int, 0>());
    step(u + 1, std::integral_constant<int, 1>());
    step(u + 2, std::integral_constant<int, 2>());
    step(u + 3, std::integral_constant<int, 3>());
    step(u + 4, std::integral_constant<int, 4>());
    step(u + 5, std::integral_constant<int, 5>());
    step(u + 6, std::integral_constant<int, 6>());
    step(u + 7, std::integral_constant<int, 7>());
    swc = sw_of(swn);
  };
  uint32_t u = 0;
  if (DX) {
    for (uint32_t quad = 1; u + 8 <= nsteps; ++quad) {
      u32x4_t nq[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) nq[t] = load_sx4(quad, t);  // past the row's end: not used
      for (int k = 1; k <= 4 && u + 8 <= nsteps; ++k, u += 8) {
        steps8(u);
#pragma unroll
        for (int t = 0; t < 4; ++t) sx[t] = k == 1 ? sxq[t][1] : k == 2 ? sxq[t][2] : sxq[t][3];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) sxq[t] = nq[t];
      if (u % 32 == 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) sx[t] = sxq[t][0];
      }
    }
  } else {
    for (; u + 8 <= nsteps; u += 8) {
      steps8(u);
#pragma unroll
      for (int t = 0; t < 4; ++t) sx[t] = sxn[t];
    }
  }
  if (u < nsteps) step(u, std::integral_constant<int, 0>());
  if (u + 1 < nsteps) step(u + 1, std::integral_constant<int, 1>());
  if (u + 2 < nsteps) step(u + 2, std::integral_constant<int, 2>());
  if (u + 3 < nsteps) step(u + 3, std::integral_constant<int, 3>());
  if (u + 4 < nsteps) step(u + 4, std::integral_constant<int, 4>());
  if (u + 5 < nsteps) step(u + 5, std::integral_constant<int, 5>());
  if (u + 6 < nsteps) step(u + 6, std::integral_constant<int, 6>());

  // (lane numbers formed anew: what is derived from them here need not live
  // through the loop, whose registers are all taken)
  int le = lane;
  asm volatile("" : "+v"(le));
  const int ge = le >> 5, ce = le & 31;
  if (p.r > 0) {
    // the next sixteen columns' fragments are loaded while one's multiply
    bf16x8_t wa[2][4], xb[2][4];
    auto load = [&](int c0, bf16x8_t(&w)[4], bf16x8_t(&x)[4]) {
#pragma unroll
      for (int f = 0; f < 4; ++f) w[f] = tail_weight(p, f0 + wf + 32 * f + ce, feats, c0 + 8 * ge);
#pragma unroll
      for (int t = 0; t < 4; ++t) x[t] = tail_token(p, t0 + wt + 32 * t + ce, c0 + 8 * ge);
    };
    auto mul = [&](const bf16x8_t(&w)[4], const bf16x8_t(&x)[4]) {
#pragma unroll
      for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int t = 0; t < 4; ++t)
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

  // every wave's copies have landed and every fragment is read before the
  // output tile goes over the stages
  dma::wait_vm<0>();
  __syncthreads();
  // lane l, value v: token 32 t + l % 32, feature 8 (v / 4) + 4 (l / 32) + v % 4
  uint16_t* out = reinterpret_cast<uint16_t*>(lds);
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int v = 0; v < 16; v += 4)
        *reinterpret_cast<uint2*>(out + (wt + 32 * t + ce) * kOutLd + wf + 32 * f + 2 * v + 4 * ge) =
            make_uint2(pack_bf16x2(acc[f][t][v], acc[f][t][v + 1]), pack_bf16x2(acc[f][t][v + 2], acc[f][t][v + 3]));
  __syncthreads();
  for (int e = threadIdx.x; e < WT * WF / 8; e += 256) {
    const int R = e >> 5, col = (e & 31) * 8;
    if (t0 + R < p.T && f0 + col < feats)
      *reinterpret_cast<u32x4_t*>(p.C + (t0 + R) * feats + f0 + col) = *reinterpret_cast<const u32x4_t*>(out + R * kOutLd + col);
  }
}

}  // namespace

hipError_t launch_fp8_wide(const Fp8Params& p, hipStream_t stream) {
  WideLaunch L{};
  L.p = p;
  L.mt = (int32_t)((p.T + WT - 1) / WT);
  L.nt = (int32_t)(((p.dx ? p.Kw : p.Nw) + WF - 1) / WF);
  L.group = 4;
  const int64_t tiles = (int64_t)L.mt * L.nt;
  KernelEvents ev(KID_FP8_GEMM);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8));
  if (p.dx) hipExtLaunchKernelGGL(k_fp8_wide<true>, grid, dim3(256), 0, stream, ev.start(), ev.stop(), 0, L);
  else hipExtLaunchKernelGGL(k_fp8_wide<false>, grid, dim3(256), 0, stream, ev.start(), ev.stop(), 0, L);
  return hipGetLastError();
}

}  // namespace qlora
