// Shared pieces of the 8-bit key/value cache: e4m3 codes with one fp32 scale for each
// block of tokens and head.
#pragma once

#include "ssd_common.cuh"

namespace ssd {

constexpr int kPageTokens = 128;          // tokens of a page

// two fp32 -> two e4m3 codes (nearest even, saturating at +-448), low byte = first
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// two e4m3 codes (low 16 bits) -> two fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

inline bool scale_block_ok(int sb) { return sb == 16 || sb == 32 || sb == 64 || sb == 128; }
inline int log2_of(int sb) { return sb == 16 ? 4 : sb == 32 ? 5 : sb == 64 ? 6 : 7; }

}  // namespace ssd
