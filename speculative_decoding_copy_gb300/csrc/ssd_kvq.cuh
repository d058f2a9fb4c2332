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

// four of them, low byte = first
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// two e4m3 codes (low 16 bits) -> two fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

__device__ __forceinline__ void e4m3x2_to_f32(uint32_t codes, float& lo, float& hi) {
  const uint32_t f = e4m3x2_to_f16x2(codes);
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(f));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// bytes [p, p + n) that a call reads or writes
struct Span {
  const void* p;
  int64_t n;
};

// whether one of the first `writes` spans shares a byte with any other
inline bool overlap(const Span* s, int writes, int count) {
  for (int i = 0; i < writes; ++i)
    for (int j = i + 1; j < count; ++j) {
      const char *a = static_cast<const char*>(s[i].p), *b = static_cast<const char*>(s[j].p);
      if (a != nullptr && b != nullptr && s[i].n > 0 && s[j].n > 0 && a < b + s[j].n && b < a + s[i].n) return true;
    }
  return false;
}

inline bool scale_block_ok(int sb) { return sb == 16 || sb == 32 || sb == 64 || sb == 128; }
inline int log2_of(int sb) { return sb == 16 ? 4 : sb == 32 ? 5 : sb == 64 ? 6 : 7; }

}  // namespace ssd
