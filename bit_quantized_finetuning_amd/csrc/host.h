// Host-side helpers shared by the C entry points: size arithmetic, alignment
// checks, workspace offsets, and the way the adapter products are split.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "kernels.h"

namespace qlora {

constexpr int64_t kMaxDim = QLORA_MAX_DIM;
constexpr int64_t kMaxTokens = QLORA_MAX_TOKENS;

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline int rank_pad(int r) { return r > 0 ? (int)ceil_div(r, 16) * 16 : 0; }

// K slices of the small-T adapter product (one tile counter per 16-token tile).
inline int lora_small_ksplit(int64_t T, int64_t K) {
  if (T > 64) return 1;
  int64_t ks = ceil_div(K, 32) / 8;
  return (int)std::max<int64_t>(1, std::min<int64_t>(ks, 64));
}

template <typename T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<uint8_t *>(ws) + off);
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

}  // namespace qlora
