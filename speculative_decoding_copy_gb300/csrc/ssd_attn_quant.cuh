// Internal interface of the attention over the 8-bit cache.
#pragma once

#include "ssd_kvq.cuh"

namespace ssd {

struct AttnQuantParams {
  const uint16_t* q;            // bf16 [B][NT][Hq][dh]
  const uint8_t* k_cache;       // e4m3
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const uint16_t* k_cand;       // bf16 [B][NT][Hkv][dh]
  const uint16_t* v_cand;
  void* out;
  const int32_t* prefix_len;
  const int32_t* blk_len;
  const int32_t* block_table;   // or null: contiguous
  int B, NB, Dmax, Hq, Hkv;
  int pages_per_seq;
  int sb_log2;                  // tokens of a scale block, log2
  int out_f32;
  float scale_log2;             // softmax scale times log2(e)
  int longest_first;            // CTAs in the order of the prefix lengths
  int64_t capacity;             // most prefix tokens
  int64_t page_tokens;          // tokens of one page, P_max of a contiguous cache
  int64_t num_pages;            // B of a contiguous cache
  int64_t blocks;               // scale blocks of a page
  WsHeader* hdr;
};

constexpr float kLeastVScaleLog2 = -100.f;     // a smaller v scale counts as this

// Own-block keys have no value scale in the exponent, so beside prefix keys of the same score
// they would look 1 / sv times as heavy, and a reference maximum set by one would push the prefix's
// probabilities, which have 8 or 16 bits, to the low end of their range. Each enters the maximum with
// the scale that a cache block of its value row alone would have, so that the reference is the
// largest contribution to the output whatever the values' size; its own probability, a bf16
// number or two, has the range for the rest. The log2 of that scale, from the largest finite
// magnitude of the row as bf16 bits; the bounds keep weights, sums and outputs in fp32's range.
__device__ __forceinline__ float own_scale_log2(uint32_t top) {
  return static_cast<float>(min(max(static_cast<int>(top >> 7) - 127 - 8, -100), 60));
}

// tensor-core path for many rows (ssd_attn_quant_tc.cu)
bool attn_quant_tc_applies(const AttnQuantParams& p);
int attn_quant_tc_launch(const AttnQuantParams& p, int dh, cudaStream_t s);

}  // namespace ssd
