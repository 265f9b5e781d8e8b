// C entry points of the operators on logits: validation and launches.  The
// declarations, with argument meaning and error behaviour, are in
// include/qlora.h.
#include "api.hpp"
#include "logits.hpp"

using namespace qlora;

namespace {

// scale * log2(e) and its product with a difference of logits stay finite or go to -inf
constexpr float kMostScale = 1.2676506e30f;  // 2^100

int64_t format_bytes(int32_t format) { return format == QLORA_W_F32 ? 4 : 2; }
bool aligned_to(const void* p, int64_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

int check_rows(int64_t T, int64_t vocab, int32_t format, int64_t ld, float scale) {
  if (format != QLORA_W_F32 && format != QLORA_W_BF16 && format != QLORA_W_F16) return QLORA_ERR_UNSUPPORTED;
  if (T < 0 || T > kLogitsMostRows || vocab <= 0 || vocab >= kMaxDim - 16 || ld < vocab || ld >= kMaxDim)
    return QLORA_ERR_SHAPE;
  if (!(scale > 0.0f) || scale > kMostScale) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

int check_grad(int64_t T, int64_t vocab, int32_t format, int64_t out_cols, int64_t out_ld) {
  if (out_cols < vocab || out_cols >= kMaxDim - 16 || out_ld < out_cols || out_ld >= kMaxDim) return QLORA_ERR_SHAPE;
  if (T > 0 && logits_grad_groups(1, out_cols, format) > kGradMostGroups / T) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

bool top_ok(int32_t top, int64_t vocab) { return top >= 0 && top <= kLogitsMost && top <= vocab; }

// The gradients' rows are the logits' own, or elsewhere.
bool in_place_ok(const void* z, int64_t ld, const void* dz, int64_t out_ld) { return z != dz || ld == out_ld; }

}  // namespace

extern "C" {

int qlora_token_logprob(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale,
                        int32_t n, const int64_t* tokens, float* logprob, float* stats, float* entropy, int32_t top,
                        int64_t* top_ids, float* top_logprob, void* stream) {
  const int st = check_rows(T, vocab, format, ld, scale);
  if (st) return st;
  if (n < 0 || n > kLogitsMost || !top_ok(top, vocab)) return QLORA_ERR_SHAPE;
  if (T > 0 && (!logits || !stats || (n > 0 && (!tokens || !logprob)) || (top > 0 && (!top_ids || !top_logprob))))
    return QLORA_ERR_NULL;
  if (!aligned_to(logits, format_bytes(format)) || !aligned_to(tokens, 8) || !aligned4(logprob) ||
      !aligned4(stats) || !aligned4(entropy) || !aligned_to(top_ids, 8) || !aligned4(top_logprob))
    return QLORA_ERR_UNSUPPORTED;
  ScoreParams P{};
  P.in = LogitsRows{logits, format, T, vocab, ld, scale};
  P.n = n; P.tokens = tokens; P.logprob = logprob; P.stats = stats; P.entropy = entropy;
  P.top = top; P.top_ids = top_ids; P.top_logprob = top_logprob;
  HIP_TRY(launch_score(P, (hipStream_t)stream));
  return QLORA_OK;
}

int qlora_token_logprob_bwd(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale,
                            int32_t n, const int64_t* tokens, const float* stats, const float* entropy,
                            const float* d_logprob, const float* d_entropy, void* dlogits, int64_t out_cols,
                            int64_t out_ld, void* stream) {
  int st = check_rows(T, vocab, format, ld, scale);
  if (!st) st = check_grad(T, vocab, format, out_cols, out_ld);
  if (st) return st;
  if (n < 0 || n > kLogitsMost) return QLORA_ERR_SHAPE;
  if (T > 0 && (!logits || !stats || !dlogits || (n > 0 && (!tokens || !d_logprob)) || (d_entropy && !entropy)))
    return QLORA_ERR_NULL;
  if (!aligned_to(logits, format_bytes(format)) || !aligned_to(dlogits, format_bytes(format)) ||
      !aligned_to(tokens, 8) || !aligned4(stats) || !aligned4(entropy) || !aligned4(d_logprob) ||
      !aligned4(d_entropy) || !in_place_ok(logits, ld, dlogits, out_ld))
    return QLORA_ERR_UNSUPPORTED;
  LogitsGradParams P{};
  P.in = LogitsRows{logits, format, T, vocab, ld, scale};
  P.n = n; P.ids = tokens; P.stats = stats; P.d_out = d_logprob; P.entropy = entropy; P.d_entropy = d_entropy;
  P.dz = dlogits; P.out_cols = out_cols; P.out_ld = out_ld;
  HIP_TRY(launch_logits_grad(P, (hipStream_t)stream));
  return QLORA_OK;
}

int qlora_distill_fwd(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale, int32_t k,
                      const int64_t* ids, const float* values, int32_t rest, float* loss, float* stats, void* stream) {
  const int st = check_rows(T, vocab, format, ld, scale);
  if (st) return st;
  if (k < 1 || k > kLogitsMost) return QLORA_ERR_SHAPE;
  if (T > 0 && (!logits || !ids || !values || !loss || !stats)) return QLORA_ERR_NULL;
  if (!aligned_to(logits, format_bytes(format)) || !aligned_to(ids, 8) || !aligned4(values) || !aligned4(loss) ||
      !aligned4(stats))
    return QLORA_ERR_UNSUPPORTED;
  DistillParams P{};
  P.in = LogitsRows{logits, format, T, vocab, ld, scale};
  P.k = k; P.ids = ids; P.values = values; P.rest = rest != 0; P.loss = loss; P.stats = stats;
 
  HIP_TRY(launch_distill(P, (hipStream_t)stream));
  return QLORA_OK;
}

int qlora_distill_bwd(int64_t T, int64_t vocab, const void* logits, int32_t format, int64_t ld, float scale, int32_t k,
                      const int64_t* ids, const float* values, int32_t rest, const float* stats, const float* d_loss,
                      void* dlogits, int64_t out_cols, int64_t out_ld, void* stream) {
  int st = check_rows(T, vocab, format, ld, scale);
  if (!st) st = check_grad(T, vocab, format, out_cols, out_ld);
  if (st) return st;
  if (k < 1 || k > kLogitsMost) return QLORA_ERR_SHAPE;
  if (T > 0 && (!logits || !ids || !values || !stats || !d_loss || !dlogits)) return QLORA_ERR_NULL;
  if (!aligned_to(logits, format_bytes(format)) || !aligned_to(dlogits, format_bytes(format)) || !aligned_to(ids, 8) ||
      !aligned4(values) || !aligned4(stats) || !aligned4(d_loss) || !in_place_ok(logits, ld, dlogits, out_ld))
    return QLORA_ERR_UNSUPPORTED;
  LogitsGradParams P{};
  P.in = LogitsRows{logits, format, T, vocab, ld, scale};
  P.n = k; P.ids = ids; P.values = values; P.distill = 1; P.rest = rest != 0; P.stats = stats; P.d_out = d_loss;
  P.dz = dlogits; P.out_cols = out_cols; P.out_ld = out_ld;
  HIP_TRY(launch_logits_grad(P, (hipStream_t)stream));
  return QLORA_OK;
}

}  // extern "C"
