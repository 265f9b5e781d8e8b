// Helpers shared by the files that hold the C entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qlora.h"

namespace qlora {

constexpr int kMaxRank = 128;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Columns of a hi/lo pair of rank r: 2r in whole multiples of 64.
inline int64_t hilo_ld(int32_t r) { return cdiv(2 * (int64_t)r, 64) * 64; }

// The kernels address every dense operand with 32-bit byte offsets (buffer
// resources capped below 2 GiB): the packed weight (or an 8-bit weight's
// codes), X, Y, dY, dX and the workspace's [T][2r] pairs must each stay below
// kMaxOperandBytes.
constexpr int64_t kMaxOperandBytes = 0x7FFFFFF0LL;
constexpr int64_t kMaxDim = (int64_t)1 << 31;

// Workspace carving: a bump allocator over the caller's buffer.
struct Carve {
  char* base;
  size_t off = 0;
  explicit Carve(void* b) : base(static_cast<char*>(b)) {}
  void* take(size_t bytes) {
    void* p = base ? base + off : nullptr;
    off += align256(bytes);
    return p;
  }
};

#define HIP_TRY(expr)                          \
  do {                                         \
    if ((expr) != hipSuccess) return QLORA_ERR_HIP; \
  } while (0)

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t stream);

// The rank-r product G = dY B (fp32 [T][r]) and the hi/lo pair of s*G into Gs
// [T][hilo_ld(r)]; part: lora_g_part_bytes of scratch.
size_t lora_g_part_bytes(int64_t T, int64_t N, int32_t r);
int lora_g(const uint16_t* dY, const uint16_t* B, int64_t T, int64_t N, int32_t r, float s, float* part,
           size_t part_bytes, float* G, uint16_t* Gs, hipStream_t st);

}  // namespace qlora
