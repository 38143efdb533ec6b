// Geometry of the 4-bit key/value cache (layout in include/slope_serving.h):
// where a token's codes and words lie inside its 16-token block.
#pragma once

#include <cstdint>

#include "slope_serving.h"

namespace slope {

constexpr int kKv4Block = 16;  // tokens of a block
constexpr int kKv4Group = 32;  // channels that share a scale and a minimum

__host__ __device__ constexpr int kv4_key_bytes(int dqk) { return kKv4Block * dqk / 2; }
__host__ __device__ constexpr int kv4_value_bytes(int dv) { return kKv4Block * dv / 2; }
__host__ __device__ constexpr int kv4_words(int dqk, int dv) { return (dqk + dv) / kKv4Group; }
__host__ __device__ constexpr int kv4_block_bytes(int dqk, int dv) {
  return kv4_key_bytes(dqk) + kv4_value_bytes(dv) + kKv4Block * 4 * kv4_words(dqk, dv);
}

// Byte offset, in the value codes, of the word that holds channels 64 * chunk + 4 * g .. + 3 (low half) and
// 64 * chunk + 32 + 4 * g .. + 3 (high half) of token t.
__host__ __device__ constexpr int kv4_value_offset(int t, int chunk, int g) {
  return (chunk * 32 + g * 4 + t % 8 / 2) * 16 + (t % 2 + 2 * (t / 8)) * 4;
}

inline bool kv4_supported(int64_t dqk, int64_t dv) {
  return (dqk == 64 || dqk == 128 || dqk == 192) && (dv == 64 || dv == 128);
}

// Argument checks of a cache (its data pointer among them).
slope_status check_kv4_cache(const slope_kv4_cache* c);

}  // namespace slope
