// C entry points of the 8-bit forms and of the linear layer on an 8-bit base
// weight: validation, workspace planning and the sequence of launches.  The
// declarations, with argument meaning and error behaviour, are in
// include/qlora.h.
#include <algorithm>

#include "api.hpp"
#include "fp8.hpp"
#include "trace.hpp"

using namespace qlora;

namespace {

int check_form(int64_t rows, int64_t cols, int32_t block_rows) {
  if (block_rows != 1 && block_rows != kFp8Block) return QLORA_ERR_UNSUPPORTED;
  if (rows < 0 || cols <= 0 || cols % 64 != 0 || rows >= kMaxDim || cols >= kMaxDim) return QLORA_ERR_SHAPE;
  // units of 512 columns are counted with 32 bits, sixteen threads each; the
  // restore's threads, sixteen codes each in workgroups of 256, are fewer than 2^32
  if (rows * (fp8_scale_ld(cols) / 4) >= (int64_t)1 << 27) return QLORA_ERR_SHAPE;
  if (rows * (cols / 16) > ((int64_t)1 << 32) - 256) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

// d_out, d_in, T and r of a layer on an 8-bit weight
int check_fp8_layer(int64_t N, int64_t K, int64_t T, int32_t r) {
  if (N <= 0 || K <= 0 || N % 64 != 0 || K % 64 != 0) return QLORA_ERR_SHAPE;
  if (T < 0 || r < 0 || r > kMaxRank) return QLORA_ERR_SHAPE;
  if (N >= kMaxDim || K >= kMaxDim || T >= kMaxDim) return QLORA_ERR_SHAPE;
  const int64_t pair = hilo_ld(r) * 2;
  if (N * K > kMaxOperandBytes || T * K * 2 > kMaxOperandBytes || T * N * 2 > kMaxOperandBytes ||
      T * pair > kMaxOperandBytes || N * pair > kMaxOperandBytes || K * pair > kMaxOperandBytes)
    return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

struct Fp8FwdWs {
  float* U = nullptr;
  uint16_t* Us = nullptr;
  uint16_t* Bp = nullptr;  // the tail's pair operand, where B cannot be read in place
  float* part = nullptr;
  size_t part_bytes = 0;
  size_t bytes = 0;
};

Fp8FwdWs plan_fwd(int64_t N, int64_t K, int64_t T, int32_t r, void* ws) {
  Fp8FwdWs w;
  Carve c(ws);
  if (T > 0) {
    w.part_bytes = fp8_product_part_bytes(T, N, K, 0, r);
    if (r > 0 && T > kFp8FewT) {
      w.U = static_cast<float*>(c.take((size_t)T * r * 4));
      w.Us = static_cast<uint16_t*>(c.take((size_t)T * hilo_ld(r) * 2));
      if (r % 8 != 0) w.Bp = static_cast<uint16_t*>(c.take((size_t)N * hilo_ld(r) * 2));
      w.part_bytes = std::max(w.part_bytes, fp8_down_part_bytes(T, K, r));
    }
    w.part = static_cast<float*>(c.take(w.part_bytes));
  }
  w.bytes = c.off;
  return w;
}

struct Fp8BwdWs {
  uint8_t* dYc = nullptr;
  uint8_t* dYs = nullptr;
  float* G = nullptr;
  float* U = nullptr;
  uint16_t* Gs = nullptr;
  uint16_t* Ap = nullptr;
  float* part = nullptr;  // of the products, which run one after another
  size_t part_bytes = 0;
  size_t bytes = 0;
};

Fp8BwdWs plan_bwd(int64_t N, int64_t K, int64_t T, int32_t r, void* ws) {
  Fp8BwdWs w;
  Carve c(ws);
  if (T > 0) {
    w.dYc = static_cast<uint8_t*>(c.take((size_t)(T * N)));
    w.dYs = static_cast<uint8_t*>(c.take((size_t)(T * fp8_scale_ld(N))));
    w.part_bytes = fp8_product_part_bytes(T, N, K, 1, r);
    if (r > 0) {
      w.G = static_cast<float*>(c.take((size_t)T * r * 4));
      w.U = static_cast<float*>(c.take((size_t)T * r * 4));
      w.Gs = static_cast<uint16_t*>(c.take((size_t)T * hilo_ld(r) * 2));
      if (T > kFp8FewT) w.Ap = static_cast<uint16_t*>(c.take((size_t)K * hilo_ld(r) * 2));
      w.part_bytes = std::max(std::max(w.part_bytes, fp8_down_part_bytes(T, K, r)),
                              std::max(lora_g_part_bytes(T, N, r), fp8_grad_part_bytes(T, K, N, r)));
      if (fp8_form_ok(r)) w.part_bytes = std::max(w.part_bytes, fp8_form_part_bytes(T, N, r));
    }
    w.part = static_cast<float*>(c.take(w.part_bytes));
  }
  w.bytes = c.off;
  return w;
}

}  // namespace

extern "C" {

int qlora_fp8_sizes(int64_t rows, int64_t cols, int32_t block_rows, size_t* codes_bytes, size_t* scales_bytes) {
  if (!codes_bytes || !scales_bytes) return QLORA_ERR_NULL;
  const int st = check_form(rows, cols, block_rows);
  if (st) return st;
  *codes_bytes = (size_t)(rows * cols);
  *scales_bytes = (size_t)(fp8_scale_rows(rows, block_rows) * fp8_scale_ld(cols));
  return QLORA_OK;
}

int qlora_quantize_fp8(int64_t rows, int64_t cols, int32_t block_rows, const void* M, int32_t m_format,
                       uint8_t* codes, uint8_t* scales, void* stream) {
  const int st = check_form(rows, cols, block_rows);
  if (st) return st;
  if (m_format != QLORA_W_F32 && m_format != QLORA_W_BF16 && m_format != QLORA_W_F16) return QLORA_ERR_UNSUPPORTED;
  if (rows > 0 && (!M || !codes || !scales)) return QLORA_ERR_NULL;
  if (!aligned16(M) || !aligned16(codes) || !aligned4(scales)) return QLORA_ERR_UNSUPPORTED;
  HIP_TRY(launch_fp8_quantize(M, m_format, rows, cols, block_rows, codes, scales, (hipStream_t)stream));
  return QLORA_OK;
}

int qlora_dequantize_fp8(int64_t rows, int64_t cols, int32_t block_rows, const uint8_t* codes, const uint8_t* scales,
                         uint16_t* M_hat, void* stream) {
  const int st = check_form(rows, cols, block_rows);
  if (st) return st;
  if (rows > 0 && (!codes || !scales || !M_hat)) return QLORA_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales) || !aligned16(M_hat)) return QLORA_ERR_UNSUPPORTED;
  HIP_TRY(launch_fp8_dequantize(codes, scales, rows, cols, block_rows, M_hat, (hipStream_t)stream));
  return QLORA_OK;
}

int qlora_fp8_fwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t T, int32_t r, size_t* bytes) {
  if (!bytes) return QLORA_ERR_NULL;
  const int st = check_fp8_layer(d_out, d_in, T, r);
  if (st) return st;
  *bytes = plan_fwd(d_out, d_in, T, r, nullptr).bytes;
  return QLORA_OK;
}

int qlora_fp8_linear_fwd(int64_t d_out, int64_t d_in, const uint8_t* W_codes, const uint8_t* W_scales, int64_t T,
                         const uint8_t* X_codes, const uint8_t* X_scales, int32_t r, float alpha, const uint16_t* A,
                         const uint16_t* B, uint16_t* Y, float* U_out, void* workspace, size_t workspace_bytes,
                         void* stream) {
  const int64_t N = d_out, K = d_in;
  const int st = check_fp8_layer(N, K, T, r);
  if (st) return st;
  if (!W_codes || !W_scales) return QLORA_ERR_NULL;
  if (T > 0 && (!X_codes || !X_scales || !Y)) return QLORA_ERR_NULL;
  if (r > 0 && (!A || !B)) return QLORA_ERR_NULL;
  if (!aligned16(W_codes) || !aligned4(W_scales) || !aligned16(X_codes) || !aligned4(X_scales) || !aligned16(A) ||
      !aligned16(B) || !aligned16(Y) || !aligned16(U_out) || !aligned16(workspace))
    return QLORA_ERR_UNSUPPORTED;
  const Fp8FwdWs w = plan_fwd(N, K, T, r, workspace);
  if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes)) return QLORA_ERR_WORKSPACE;
  if (T == 0) return QLORA_OK;
  hipStream_t s_ = (hipStream_t)stream;
  Fp8Params P{};
  P.X = X_codes; P.Xs = X_scales; P.W = W_codes; P.Ws = W_scales;
  P.T = T; P.Nw = N; P.Kw = K; P.dx = 0; P.r = r; P.ldh = hilo_ld(r);
  P.C = Y; P.part = w.part; P.part_bytes = w.part_bytes;
  if (r > 0) P.s = alpha / (float)r;
  if (r > 0 && T <= kFp8FewT) {
    P.A = A; P.M = B; P.U = U_out;
  } else if (r > 0) {
    const Fp8DownParams Dn{X_codes, X_scales, A, T, K, r, P.s, U_out ? U_out : w.U, w.Us, P.ldh, w.part, w.part_bytes};
    HIP_TRY(launch_fp8_down(Dn, s_));
    P.At = w.Us;
    P.Bt = B;
    if (w.Bp) {
      HIP_TRY(launch_fp8_pair(B, N, r, P.ldh, 0, w.Bp, s_));
      P.Bt = w.Bp;
      P.bt_pair = 1;
    }
  }
  HIP_TRY(launch_fp8_product(P, s_));
  return QLORA_OK;
}

int qlora_fp8_bwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t T, int32_t r, size_t* bytes) {
  if (!bytes) return QLORA_ERR_NULL;
  const int st = check_fp8_layer(d_out, d_in, T, r);
  if (st) return st;
  *bytes = plan_bwd(d_out, d_in, T, r, nullptr).bytes;
  return QLORA_OK;
}

int qlora_fp8_linear_bwd(int64_t d_out, int64_t d_in, const uint8_t* W_codes, const uint8_t* W_scales, int64_t T,
                         const uint8_t* X_codes, const uint8_t* X_scales, int32_t r, float alpha, const uint16_t* A,
                         const uint16_t* B, const float* U_in, const uint16_t* dY, uint16_t* dX, float* dA, float* dB,
                         int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t N = d_out, K = d_in;
  const int st = check_fp8_layer(N, K, T, r);
  if (st) return st;
  if (!W_codes || !W_scales) return QLORA_ERR_NULL;
  if (T > 0 && (!dY || (r > 0 && (!X_codes || !X_scales)))) return QLORA_ERR_NULL;
  if (r > 0 && (!A || !B || !dA || !dB)) return QLORA_ERR_NULL;
  if (!aligned16(W_codes) || !aligned4(W_scales) || !aligned16(X_codes) || !aligned4(X_scales) || !aligned16(A) ||
      !aligned16(B) || !aligned16(U_in) || !aligned16(dY) || !aligned16(dX) || !aligned16(dA) || !aligned16(dB) ||
      !aligned16(workspace))
    return QLORA_ERR_UNSUPPORTED;
  const Fp8BwdWs w = plan_bwd(N, K, T, r, workspace);
  if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes)) return QLORA_ERR_WORKSPACE;
  hipStream_t s_ = (hipStream_t)stream;
  if (T == 0) {
    if (r > 0 && !accumulate) {
      HIP_TRY(launch_fill_zero(dA, (int64_t)r * K, s_));
      HIP_TRY(launch_fill_zero(dB, N * r, s_));
    }
    return QLORA_OK;
  }
  const float s = r > 0 ? alpha / (float)r : 0.0f;
  const int64_t ldh = hilo_ld(r);
  const bool form = fp8_form_ok(r);  // G and, for dX, the 8-bit form of dY from one pass over it
  const float* U = U_in;
  if (r > 0) {
    if (!U) {
      const Fp8DownParams Dn{X_codes, X_scales, A, T, K, r, s, w.U, nullptr, ldh, w.part, w.part_bytes};
      HIP_TRY(launch_fp8_down(Dn, s_));
      U = w.U;
    }
    if (form) {
      const Fp8FormParams F{dY, B, T, N, r, s, dX ? w.dYc : nullptr, w.dYs, w.G, w.Gs, ldh, w.part, w.part_bytes};
      HIP_TRY(launch_fp8_form(F, s_));
    } else {
      const int e = lora_g(dY, B, T, N, r, s, w.part, w.part_bytes, w.G, w.Gs, s_);
      if (e) return e;
    }
  }
  if (dX) {
    if (!form) HIP_TRY(launch_fp8_quantize(dY, QLORA_W_BF16, T, N, 1, w.dYc, w.dYs, s_));
    Fp8Params P{};
    P.X = w.dYc; P.Xs = w.dYs; P.W = W_codes; P.Ws = W_scales;
    P.T = T; P.Nw = N; P.Kw = K; P.dx = 1; P.r = r; P.ldh = ldh;
    P.C = dX; P.part = w.part; P.part_bytes = w.part_bytes;
    if (r > 0 && T <= kFp8FewT) {
      P.s = s; P.M = A; P.G = w.G;
    } else if (r > 0) {
      HIP_TRY(launch_fp8_pair(A, K, r, ldh, 1, w.Ap, s_));
      P.At = w.Gs; P.Bt = w.Ap; P.bt_pair = 1;
    }
    HIP_TRY(launch_fp8_product(P, s_));
  }
  if (r > 0) {
    const Fp8GradParams Gr{X_codes, X_scales, dY, w.G, U, T, K, N, r, s, dA, dB, accumulate != 0, w.part, w.part_bytes};
    HIP_TRY(launch_fp8_grad(Gr, s_));
  }
  return QLORA_OK;
}

}  // extern "C"
