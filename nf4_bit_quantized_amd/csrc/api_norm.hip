// C entry points of the residual norm: validation and launches.  The
// declarations, with argument meaning and error behaviour, are in
// include/qlora.h.
#include <cmath>

#include "api.hpp"
#include "norm.hpp"

using namespace qlora;

namespace {

int check_norm(int64_t T, int64_t D, int32_t stream_format, int32_t weight_format, float eps, float scale) {
  if (T < 0 || T > kNormMostRows || D <= 0 || D % 64 != 0 || D > kNormMostCols) return QLORA_ERR_SHAPE;
  if (stream_format != QLORA_W_F32 && stream_format != QLORA_W_BF16) return QLORA_ERR_UNSUPPORTED;
  if (weight_format != QLORA_W_F32 && weight_format != QLORA_W_BF16) return QLORA_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(scale)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

bool all16(std::initializer_list<const void*> p) {
  for (const void* q : p)
    if (!aligned16(q)) return false;
  return true;
}

}  // namespace

extern "C" {

int qlora_norm_fwd(int64_t T, int64_t D, const void* h, int32_t stream_format, const uint16_t* block,
                   const void* weight, const void* post_weight, const void* gate, int32_t weight_format, float scale,
                   float eps, void* h_out, uint16_t* X, uint8_t* codes, uint8_t* scales, float* stats, void* stream) {
  const int st = check_norm(T, D, stream_format, weight_format, eps, scale);
  if (st) return st;
  if (!weight) return QLORA_ERR_NULL;
  if (T > 0 && ((!block && (post_weight || gate)) || !codes != !scales)) return QLORA_ERR_NULL;
  if (T > 0 && (!h || !stats || (block && !h_out) || (!X && !codes))) return QLORA_ERR_NULL;
  if (!all16({h, block, weight, post_weight, gate, h_out, X, codes}) || !aligned4(scales) || !aligned4(stats))
    return QLORA_ERR_UNSUPPORTED;
  NormParams P{};
  P.T = T; P.D = (int)D; P.stream = stream_format; P.weights = weight_format; P.eps = eps; P.scale = scale;
  P.h = h; P.block = block; P.weight = weight; P.post_weight = post_weight; P.gate = gate;
  P.h_out = h_out; P.x = X; P.codes = codes; P.scales = scales; P.stats = stats;
  HIP_TRY(launch_norm(P, (hipStream_t)stream));
  return QLORA_OK;
}

int qlora_norm_bwd_workspace_bytes(int64_t T, int64_t D, size_t* bytes) {
  if (!bytes) return QLORA_ERR_NULL;
  const int st = check_norm(T, D, QLORA_W_F32, QLORA_W_F32, 0.0f, 1.0f);
  if (st) return st;
  *bytes = norm_bwd_part_bytes(T, D);
  return QLORA_OK;
}

int qlora_norm_bwd(int64_t T, int64_t D, const uint16_t* dX, const void* h_out, int32_t stream_format,
                   const uint16_t* block, const void* weight, const void* post_weight, const void* gate,
                   int32_t weight_format, float scale, const float* stats, const void* dh_out, void* dh,
                   uint16_t* dblock, float* dweight, float* dpost_weight, float* dgate, int32_t accumulate,
                   void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_norm(T, D, stream_format, weight_format, 0.0f, scale);
  if (st) return st;
  if (!weight || (T > 0 && !block && (post_weight || gate))) return QLORA_ERR_NULL;
  if (dweight && (!post_weight != !dpost_weight || !gate != !dgate)) return QLORA_ERR_NULL;
  if (!dweight && (dpost_weight || dgate)) return QLORA_ERR_NULL;
  if (T > 0 && (!dX || !h_out || !stats || !dh || (block && !dblock))) return QLORA_ERR_NULL;
  if (!all16({dX, h_out, block, weight, post_weight, gate, dh_out, dh, dblock, dweight, dpost_weight, dgate, workspace}) ||
      !aligned4(stats))
    return QLORA_ERR_UNSUPPORTED;
  const size_t need = dweight ? norm_bwd_part_bytes(T, D) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return QLORA_ERR_WORKSPACE;
  hipStream_t s_ = (hipStream_t)stream;
  if (T == 0) {
    if (!accumulate)
      for (float* p : {dweight, dpost_weight, dgate})
        if (p) HIP_TRY(launch_fill_zero(p, D, s_));
    return QLORA_OK;
  }
  NormParams P{};
  P.T = T; P.D = (int)D; P.stream = stream_format; P.weights = weight_format; P.scale = scale;
  P.block = block; P.weight = weight; P.post_weight = post_weight; P.gate = gate;
  P.h_out = const_cast<void*>(h_out); P.stats = const_cast<float*>(stats);
  P.dx = dX; P.dh_out = dh_out; P.dh = dh; P.dblock = block ? dblock : nullptr;
  P.dweight = dweight; P.dpost_weight = dpost_weight; P.dgate = dgate; P.accumulate = accumulate != 0;
  P.part = static_cast<float*>(workspace);
  HIP_TRY(launch_norm_bwd(P, s_));
  return QLORA_OK;
}

}  // extern "C"
