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
// they look 1 / sv times as heavy, and a reference maximum set by one would push the prefix's
// probabilities, which have 8 or 16 bits, to the low end of their range. They enter the maximum
// lowered by this (log2); their own probabilities, bf16 numbers, may then pass the reference.
constexpr float kOwnLowered = 16.f;

// tensor-core path for many rows (ssd_attn_quant_tc.cu)
bool attn_quant_tc_applies(const AttnQuantParams& p);
int attn_quant_tc_launch(const AttnQuantParams& p, int dh, cudaStream_t s);

}  // namespace ssd
