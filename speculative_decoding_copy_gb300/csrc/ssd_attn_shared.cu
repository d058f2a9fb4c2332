// Verification attention of a batch whose sequences share a prompt: the prompt's keys once for all.
//
// For a present token t of sequence b and a q-head, with the row's softmax kept as (m, l, O) = (reference
// maximum, sum of 2^(s - m), sum of 2^(s - m) v) over any part of its keys, two parts join by
//   M = max(m1, m2),  l = l1 2^(m1 - M) + l2 2^(m2 - M),  O likewise,
// so the parts may be computed wherever that is cheapest: the shared prompt with the present tokens of
// all sequences as the rows of one product, a sequence's own prefix with its tokens, the own block
// (at most 256 keys) row by row. Three kernels:
//   k_plan    one CTA: list of the present tokens, offsets of the sequences, and the work in units of
//             128 keys x 128 packed rows (a row tile; two of the same keys are a "pair") x one kv head;
//   k_parts   one CTA an SM: an equal run of units each, so that a long prompt, many short prefixes or
//             both fill the GPU whatever their sizes. Where a run crosses from one pair (and head) to
//             the next, a segment ends and its (m, l, O) go to the workspace;
//   k_join    a warp a row: the segments of its shared and own keys, and its own block.
// k_parts, 576 threads, all 512 columns of TMEM: warps 0-7 and 8-15 hold a row tile each (two threads a row,
// 64 of a tile's 128 keys each): scores from TMEM into registers, the row's maximum between the two
// threads, P as bf16 pairs back into TMEM, O rescaled in TMEM only when a maximum grew by
// more than 2^8; warp 16 fetches K and V tiles by TMA into a ring of five; warp 17 issues the products,
// those of one tile while the other's softmax runs, and before that zeroes the value rows behind a
// length (0 times NaN is NaN).
// The order of a unit's products is S0 S1 | S0' PV0 S1' PV1 | ..: the next scores are issued before this
// tile's probabilities are made, so neither the products nor the exponentials wait for the other's latency.
// Segments of one row tile (few tokens) run two side by side, one in each row tile's place.
// Every wait is bounded; after one that gave up the CTA records SSD_ERR_TIMEOUT, waits (bounded) for its
// copies and products in flight and ends; rows it shares come out NaN.
//
// What bounds it (clocks of 128 keys x 256 rows, dh 128): 3350, of which the four products take 2060 at their
// best and the exponentials 1030 (8 a clock and scheduler), so it waits: in the serving batch below a CTA
// takes 657 thousand clocks for 165 such units and its segments' ends; the products are 341 thousand of
// them (tensor pipe 50% busy), their warp waits 42 for keys, 39 for scores to be read, 34 for P, 19 for
// values, 12 for Q, and a softmax warp 320 for scores. In steps: 4450 with one thread issuing in a diverged
// warp (170 clocks a product instead of 64); 3400 issued by a converged one; the same with a cubic for 3 of 8
// exponentials and with two threads a row; 3350 with the scores ahead. A segment's end (O out, the
// next Q in) costs 8000 clocks, 15000 before its rows were written side by side. 32 sequences, 9 blocks of
// 16 tokens (30% there) behind 16384 shared and up to 2048 own keys: 403-426 us, 0.5 of the bf16 rate;
// 64 single tokens behind 8192 and up to 500: 46 us for 103 MB. Head dim 64: 329 and 36 us.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "ssd_kvq.cuh"
#include "ssd_tc.cuh"

namespace ssd {
namespace shr {

using namespace tc;

constexpr int kTile = 128;                 // keys of a tile, packed rows of a row tile
constexpr int kThreads = 576;
constexpr int kSlots = 5;                  // ring of K and V tiles
constexpr int kBarBytes = 3 * 1024;
constexpr int kSegs = 20;                  // segments a CTA has described at once
constexpr int kMaxBatch = 4096;            // sequences: their offsets fit the ring before it is used
constexpr unsigned long long kWaitClocks = 1ull << 32;

// Where the segments of the shared or of the own keys go: of each (reference maximum, sum) of its rows and O, for
// `tiles` row tiles of `rows` rows, of which there are no more than the most tokens a segment can have need
struct Slots {
  float* ml;                               // [segments][tiles][rows][2]
  float* o;                                // [segments][tiles][dh / 4][rows][4]
  int tiles, rows;
  __host__ __device__ int64_t first(int64_t id, int tile) const { return (id * tiles + tile) * rows; }     // row of all segments'
};

struct Params {
  const void *q, *k_shared, *v_shared, *k_cache, *v_cache, *k_cand, *v_cand;
  void* out;
  const int32_t *shared_len, *prefix_len, *blk_len, *shared_table, *block_table;
  int B, NB, Dmax, Hq, Hkv, G;
  int tokens;                              // of a row tile: 128 / G
  int64_t S_max, P_max, num_pages;
  int shared_pages, pages_per_seq;
  float scale_log2;
  int out_f32, ctas;
  WsHeader* hdr;
  int32_t* plan;                           // kPlan numbers
  int32_t* tok;                            // the present tokens b * NT + t
  int32_t *tok_first, *unit0, *ph0, *own_len;      // [B + 1] (own_len [B])
  Slots shared, own;
};
// Work is measured in units of 1700 clocks, what a key tile takes with one row tile beside another segment's;
// with two row tiles (3400) it counts as two, and Q in and O out of a pair and head as two more tiles.
constexpr int kSetup = 2;
enum { kTokens = 0, kShare = 1, kUnits = 2, kSharedLen = 3, kSharedUnits = 4, kPlan = 16 };

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
// units of a key tile for rows of `tokens` tokens, of which a row tile holds `per`
__device__ __forceinline__ int tile_units(int tokens, int per) { return tokens > per ? 2 : 1; }

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;

// exclusive sums of three numbers over the CTA, and the totals
__device__ __forceinline__ void plan_scan(int (&v)[3], int (*part)[32], int (&total)[3]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int x[3] = {v[0], v[1], v[2]}, w[3];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += y;
    }
  __syncthreads();
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) part[k][wid] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) w[k] = part[k][lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, w[k], o);
      if (lane >= o) w[k] += y;
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    total[k] = __shfl_sync(0xffffffffu, w[k], 31);
    const int before = __shfl_sync(0xffffffffu, w[k], max(wid - 1, 0));
    v[k] = x[k] - v[k] + (wid > 0 ? before : 0);
  }
}

// Segment (of pair-and-head ph, cut by CTA c's run) has the number ph + c: from one segment to the next
// one of the two grows or both do. Pairs of the shared prompt come first, then those of each sequence
// (unit0 and ph0 count from the first of these, and so do their segments).
__global__ void __launch_bounds__(kPlanThreads) k_plan(Params p) {
  __shared__ int part[3][32];
  __shared__ int first[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int S = __ldg(p.shared_len);
  const int64_t s_cap = p.shared_table != nullptr ? 128LL * p.shared_pages : p.S_max;
  const int64_t p_cap = p.block_table != nullptr ? 128LL * p.pages_per_seq : p.P_max;
  const int pair = 2 * p.tokens;
  int tokens = 0, units = 0, ph = 0, two = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int v[3] = {0, 0, 0}, total[3];
    if (b < p.B) {
      int P = __ldg(p.prefix_len + b);
      for (int k = 0; k < p.NB; ++k) v[0] += min(max(__ldg(p.blk_len + static_cast<int64_t>(b) * p.NB + k), 0), p.Dmax);
      if (P < 0 || P > p_cap) {
        record_error(p.hdr, SSD_ERR_DEVICE, 602);
        P = 0;
      }
      p.own_len[b] = P;
      v[1] = P > 0 ? ceil_div(v[0], pair) * p.Hkv : 0;
      v[2] = v[1] * (ceil_div(P, kTile) + kSetup) * tile_units(v[0], p.tokens);
      if (v[2] > 0 && v[0] > p.tokens) two = 1;
    }
    plan_scan(v, part, total);
    first[tid] = tokens + v[0];
    if (b < p.B) {
      p.tok_first[b] = tokens + v[0];
      p.ph0[b] = ph + v[1];
      p.unit0[b] = units + v[2];
    }
    tokens += total[0];
    ph += total[1];
    units += total[2];
    __syncthreads();
    // their tokens: a warp a sequence
    for (int b = b0 + wid; b < min(p.B, b0 + kPlanThreads); b += kPlanThreads / 32) {
      int at = first[b - b0];
      for (int k0 = 0; k0 < p.NB; k0 += 32) {
        const int len = k0 + lane < p.NB ? min(max(__ldg(p.blk_len + static_cast<int64_t>(b) * p.NB + k0 + lane), 0), p.Dmax) : 0;
        for (int k = k0; k < min(p.NB, k0 + 32); ++k) {
          const int n = __shfl_sync(0xffffffffu, len, k - k0);
          for (int d = lane; d < n; d += 32) p.tok[at + d] = (b * p.NB + k) * p.Dmax + d;
          at += n;
        }
      }
    }
  }
  two = __syncthreads_or(two);
  if (tid == 0) {
    if (S < 0 || S > s_cap) {
      record_error(p.hdr, SSD_ERR_DEVICE, 601);
      S = 0;
    }
    const int ph_s = S > 0 ? ceil_div(tokens, pair) * p.Hkv : 0;
    const int units_s = ph_s * (ceil_div(S, kTile) + kSetup) * tile_units(tokens, p.tokens);
    if (units_s > 0 && tokens > p.tokens) two = 1;
    p.tok_first[p.B] = tokens;
    p.unit0[p.B] = units;
    p.plan[kTokens] = tokens;
    // (never less than a tile: a run in the middle of a pair then has one at least)
    p.plan[kShare] = max(two ? 2 : 1, ceil_div(units_s + units, p.ctas));
    p.plan[kUnits] = units_s + units;
    p.plan[kSharedLen] = S;
    p.plan[kSharedUnits] = units_s;
  }
}

// ------------------------------------------------------------------ segments
struct Seg {
  int b;                                   // sequence, or -1: the shared prompt
  int kvh, tok0, ntok;                     // first present token and their number (up to two tiles')
  int j0, j1, len;                         // key tiles, and the length of all keys
  int id;
};

// the sequence whose units hold u (unit0 ascending; the last one that starts at or before u and has any)
__device__ __forceinline__ int find_seq(const int* unit0, int B, int u) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (unit0[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// Segments of units [u, u1) for CTA c, as many as fit; returns the unit behind them. `b` is the sequence
// that u lies in, where it is not in the shared part (-1: not looked for yet).
__device__ int describe(const Params& p, Seg* segs, int* count, int c, int u, int u1, const int* unit0, const int* ph0, const int* tok_first,
                        const int* own_len, int tokens, int shared_len, int own0) {
  const int pair = 2 * p.tokens;
  int n = 0, b = -1;
  while (u < u1 && n < kSegs) {
    Seg s;
    int base, first, all, ph;
    if (u < own0) {
      s.b = -1;
      s.len = shared_len;
      base = 0;
      first = 0;
      all = tokens;
      ph = 0;
    } else {
      if (b < 0) b = find_seq(unit0, p.B, u - own0);
      while (own0 + unit0[b + 1] <= u) ++b;
      s.b = b;
      s.len = own_len[b];
      base = own0 + unit0[b];
      first = tok_first[b];
      all = tok_first[b + 1] - first;
      ph = ph0[b];
    }
    const int w = tile_units(all, p.tokens), kt = (ceil_div(s.len, kTile) + kSetup) * w, at = (u - base) / kt;
    s.kvh = at % p.Hkv;
    const int pr = at / p.Hkv;
    s.tok0 = first + pr * pair;
    s.ntok = min(pair, all - pr * pair);
    // key tile j has the w units from base + at kt + (kSetup + j) w on, and belongs to the run that has the first
    const int from = u - base - at * kt, to = min(kt, from + (u1 - u));
    s.j0 = max(ceil_div(from, w) - kSetup, 0);
    s.j1 = ceil_div(to, w) - kSetup;
    s.id = ph + at + c;
    if (s.j1 > s.j0) segs[n++] = s;
    u += to - from;
  }
  *count = n;
  return u;
}

// Segments are worked through in groups: one of two row tiles, which share its keys, or up to two of one row
// tile each, side by side, each with its own keys. Segment i begins one; returns how many it has.
__device__ __forceinline__ int group_of(const Params& p, const Seg* segs, int i, int nseg) {
  return segs[i].ntok <= p.tokens && i + 1 < nseg && segs[i + 1].ntok <= p.tokens ? 2 : 1;
}
// What row tile t of the CTA does in the group of segment i: a segment (or -1), and which of its row tiles
struct Part {
  int seg, tile;
};
__device__ __forceinline__ Part part_of(const Params& p, const Seg* segs, int i, int n, int t) {
  if (n == 2) return {i + t, 0};
  if (t == 0 || segs[i].ntok > p.tokens) return {i, t};
  return {-1, 0};
}

// row of the K or V tensor (rows of dh elements) at which key tile j of a segment starts
__device__ __forceinline__ int64_t tile_row(const Params& p, const Seg& s, int j) {
  if (s.b < 0 && p.shared_table == nullptr) return static_cast<int64_t>(s.kvh) * p.S_max + j * kTile;
  if (s.b >= 0 && p.block_table == nullptr) return (static_cast<int64_t>(s.b) * p.Hkv + s.kvh) * p.P_max + j * kTile;
  int pg = s.b < 0 ? __ldg(p.shared_table + j) : __ldg(p.block_table + static_cast<int64_t>(s.b) * p.pages_per_seq + j);
  if (pg < 0 || pg >= p.num_pages) {
    record_error(p.hdr, SSD_ERR_DEVICE, 603);
    pg = 0;
  }
  return (static_cast<int64_t>(pg) * p.Hkv + s.kvh) * kTile;
}

// ------------------------------------------------------------------ parts, tensor cores
struct Bars {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], q_full[2], o_free[2], max_read[2];
  uint64_t last;
  uint32_t tmem_base;
  int failed, count, next;
  float pair[2][256];                      // of each row tile: a maximum (at the end a sum) of every thread, for the row's other one
  Seg segs[kSegs];
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers and segments");

template <int DH>
struct Shape {
  static constexpr uint32_t kHalves = DH / 64;
  static constexpr uint32_t kHalf = kTile * 128;            // 128 rows x 64 bf16, 128-byte swizzle
  static constexpr uint32_t kTileB = kHalves * kHalf;
  static constexpr uint32_t OFF_Q = 0;                      // two row tiles
  static constexpr uint32_t OFF_RING = 2 * kTileB;
  static constexpr uint32_t OFF_BAR = OFF_RING + kSlots * kTileB;
  static constexpr uint32_t kSmem = OFF_BAR + kBarBytes;    // the base is 1024-byte aligned: there is no static shared memory
};
static_assert(Shape<128>::kSmem <= 232448, "shared memory per CTA");
static_assert(4 * (kMaxBatch + 1) * 4 <= kSlots * static_cast<int>(Shape<64>::kTileB), "offsets fit the ring");
// TMEM columns: one buffer of scores, taken by the row tiles in turns (it is free as soon as the scores are in
// registers, long before their P is made), P of tile 0 and 1 as bf16 pairs, O of tile 0 and 1
// (P in the first half of its own S, with a buffer of scores for each row tile, would fill the 512 columns too: not tried)
constexpr uint32_t TM_S = 0, TM_P = 128, TM_O = 256;

__device__ __forceinline__ bool wait(Bars& bars, uint64_t* bar, uint32_t parity, WsHeader* hdr, int where) {
  return mbar_wait_bounded(bar, parity, &bars.failed, hdr, where, kWaitClocks);
}
// without a look at `failed`: for what is in flight after a wait gave up
__device__ __forceinline__ void wait_anyway(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = clock64();
  while (!mbar_probe(bar, parity) && clock64() - t0 < kWaitClocks) {
  }
}

// two fp32 numbers in one register pair, one instruction for both
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 two(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void apart(f32x2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
k_parts(const __grid_constant__ CUtensorMap map_ks, const __grid_constant__ CUtensorMap map_vs, const __grid_constant__ CUtensorMap map_k,
        const __grid_constant__ CUtensorMap map_v, Params p) {
  using Sh = Shape<DH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = smem_u32(smem);
  Bars& bars = *reinterpret_cast<Bars*>(smem + Sh::OFF_BAR);
  // (by a shuffle: the compiler then knows it, and what follows from it, to be the same for the warp)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, cta = blockIdx.x;
  if ((sbase & 1023) != 0) {               // swizzled tiles need it
    if (tid == 0) record_error(p.hdr, SSD_ERR_DEVICE, 604);
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.s_free[t], 256);
      mbar_init(&bars.p_full[t], 256);
      mbar_init(&bars.pv_done[t], 1);
      mbar_init(&bars.q_full[t], 256);
      mbar_init(&bars.max_read[t], 256);
      mbar_init(&bars.o_free[t], 256);
    }
    mbar_init(&bars.last, 1);
    bars.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    if (lane == 0) {
      prefetch_tmap(&map_ks);
      prefetch_tmap(&map_vs);
      prefetch_tmap(&map_k);
      prefetch_tmap(&map_v);
    }
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem_base)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem_base, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the plan
  const int share = __ldcg(p.plan + kShare), units = __ldcg(p.plan + kUnits), tokens = __ldcg(p.plan + kTokens);
  const int shared_len = __ldcg(p.plan + kSharedLen);
  const int64_t start = static_cast<int64_t>(cta) * share;
  int u = static_cast<int>(start < units ? start : units);
  const int u1 = static_cast<int>(start + share < units ? start + share : units);

  // phases, each role its own: ring entries so far; of the softmax warps the tiles so far; of the
  // products one bit a row tile
  int last = -1;                                            // tile of the last scores
  uint32_t it = 0, tiles = 0, ph_s = 0, ph_p = 0, ph_q = 0, ph_o = 0, used = 0;

  bool gave_up = false;
  while (u < u1) {
    // offsets of the sequences into the ring, then this CTA's segments from there (after a wait that gave up
    // copies may still arrive in the ring)
    int* off = reinterpret_cast<int*>(smem + Sh::OFF_RING);
    for (int i = tid; i <= p.B && !gave_up; i += kThreads) {
      off[i] = __ldcg(p.unit0 + i);
      off[(p.B + 1) + i] = i < p.B ? __ldcg(p.ph0 + i) : 0;
      off[2 * (p.B + 1) + i] = __ldcg(p.tok_first + i);
      off[3 * (p.B + 1) + i] = i < p.B ? __ldcg(p.own_len + i) : 0;
    }
    __syncthreads();
    if (tid == 0)
      bars.next = describe(p, bars.segs, &bars.count, cta, u, u1, gave_up ? p.unit0 : off, gave_up ? p.ph0 : off + (p.B + 1),
                           gave_up ? p.tok_first : off + 2 * (p.B + 1), gave_up ? p.own_len : off + 3 * (p.B + 1), tokens, shared_len,
                           __ldcg(p.plan + kSharedUnits));
    fence_async_smem();                                     // TMA writes over what was just read
    __syncthreads();
    u = bars.next;
    const int nseg = bars.count;

    if (gave_up) {
      // segments that nothing computes: their rows come out NaN, not as what the workspace held
      for (int i = 0; i < nseg; ++i) {
        const Slots& w = bars.segs[i].b < 0 ? p.shared : p.own;
        for (int e = tid; e < w.tiles * w.rows; e += kThreads)
          *reinterpret_cast<float2*>(w.ml + (w.first(bars.segs[i].id, 0) + e) * 2) = make_float2(NAN, NAN);
      }
    } else if (warp < 16) {
      // -------------------------------------------------------- softmax rows: two threads a row
      const int t = warp >> 3, half = (warp >> 2) & 1;      // row tile; keys 0-63 or 64-127 of a key tile
      const int r = (warp & 3) * 32 + lane;                 // this thread's row
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t sc = tmem + TM_S + 64 * half + lane_off, pc = tmem + TM_P + 64 * t + 32 * half + lane_off;
      const uint32_t oc = tmem + TM_O + t * 128 + half * (DH / 2) + lane_off;
      auto tile_sync = [&] { asm volatile("bar.sync %0, 256;" ::"r"(1 + t) : "memory"); };
      // rows of tile t of a segment: G heads of each of its tokens; a warp brings sixteen, whose token a
      // lane knows (asked for a segment ahead)
      const int w0 = (warp & 7) * 16;
      auto rows_of = [&](const Seg& s, int tile) { return min(p.tokens, s.ntok - tile * p.tokens) * p.G; };
      auto token_of = [&](const Part& a) {
        const Seg& s = bars.segs[a.seg];
        const int mine = w0 + (lane & 15);
        return mine < rows_of(s, a.tile) ? __ldcg(p.tok + s.tok0 + a.tile * p.tokens + mine / p.G) : -1;
      };
      // the next part of this row tile behind group i (moved on), seg < 0: none
      auto next_part = [&](int& i) {
        Part a = {-1, 0};
        while (i < nseg && a.seg < 0) {
          const int n = group_of(p, bars.segs, i, nseg);
          a = part_of(p, bars.segs, i, n, t);
          i += n;
        }
        return a;
      };
      auto load_q = [&](const Seg& s, int token) {
        constexpr int CH = DH / 8;                          // 16-byte pieces of a row
        constexpr int RI = 32 / CH;                         // rows of one round
        uint4 v[16 / RI];
#pragma unroll
        for (int i = 0; i < 16 / RI; ++i) {
          const int rr = i * RI + lane / CH;
          const int tk = __shfl_sync(0xffffffffu, token, rr);
          v[i] = make_uint4(0, 0, 0, 0);
          if (tk >= 0)
            v[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                        (static_cast<int64_t>(tk) * p.Hq + s.kvh * p.G + (w0 + rr) % p.G) * DH) + lane % CH);
        }
#pragma unroll
        for (int i = 0; i < 16 / RI; ++i) {
          const int rr = w0 + i * RI + lane / CH, ch = lane % CH;
          *reinterpret_cast<uint4*>(smem + Sh::OFF_Q + t * Sh::kTileB + (ch >> 3) * Sh::kHalf + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v[i];
        }
        fence_async_smem();
        mbar_arrive(&bars.q_full[t]);
      };
      int i = 0;
      Part now = next_part(i);
      if (now.seg >= 0) load_q(bars.segs[now.seg], token_of(now));
      while (now.seg >= 0) {
        const Seg s = bars.segs[now.seg];
        const Part then = next_part(i);
        const int token = then.seg >= 0 ? token_of(then) : -1;
        float m = -INFINITY, l = 0.f;
        for (int j = s.j0; j < s.j1; ++j) {
          wait(bars, &bars.s_full[t], tiles & 1, p.hdr, 610);
          tc_fence_after();
          uint32_t v[64];
          tmem_ld32(sc, v);
          tmem_ld32(sc + 32, v + 32);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(&bars.s_free[t]);
          const int hi = s.len - j * kTile - 64 * half;
          if (hi < 64) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= hi) v[c] = 0xff800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
          // (the other threads have read the last tile's: long since, as a rule)
          if (tiles > 0) wait(bars, &bars.max_read[t], (tiles - 1) & 1, p.hdr, 613);
          float* pair = bars.pair[t];
          pair[half * 128 + r] = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          tile_sync();
          const float top = fmaxf(pair[r], pair[128 + r]) * p.scale_log2;
          mbar_arrive(&bars.max_read[t]);
          // the reference moves only when the maximum grows by more than 2^8
          const bool need = top > m + 8.f || m == -INFINITY;
          const float ref = need ? fmaxf(m, top) : m;
          const float alpha = need && m > -INFINITY ? ex2_approx(m - ref) : 1.f;     // nothing counted yet: O and l are 0
          const float sub = ref > -INFINITY ? ref : 0.f;    // every key at -inf: all weights 0
          f32x2 rs[2] = {two(0.f, 0.f), two(0.f, 0.f)};
          const f32x2 slope = two(p.scale_log2, p.scale_log2), shift = two(-sub, -sub);
          // P of keys 64 half .. + 63 as bf16 pairs
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float e0, e1;
            apart(fma2(two(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), slope, shift), e0, e1);
            const uint32_t w = pack_bf16(ex2_approx(e0), ex2_approx(e1));
            rs[(c >> 1) & 1] = add2(rs[(c >> 1) & 1], two(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
            v[c >> 1] = w;
          }
          // the product before has read the last P, and O holds the sum up to it
          if (tiles > 0) {
            wait(bars, &bars.pv_done[t], (tiles - 1) & 1, p.hdr, 611);
            tc_fence_after();
          }
          tmem_st32(pc, v);
          float sum0, sum1;
          apart(add2(rs[0], rs[1]), sum0, sum1);
          if (j > s.j0) {
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll 1
              for (int c = 0; c < DH / 64; ++c) {
                uint32_t o[32];
                tmem_ld32(oc + 32 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(oc + 32 * c, o);
              }
            }
          }
          l = l * alpha + (sum0 + sum1);
          m = ref;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars.p_full[t]);
          ++tiles;
        }
        // the last scores are read: Q is free for the next segment, whose first product may start
        if (then.seg >= 0) load_q(bars.segs[then.seg], token);
        tile_sync();                                        // the last maxima are read
        float* sums = bars.pair[t];
        if (half == 1) sums[r] = l;
        tile_sync();
        const float l_other = sums[r];
        wait(bars, &bars.pv_done[t], (tiles - 1) & 1, p.hdr, 612);
        tc_fence_after();
        const int nrow = rows_of(s, now.tile);
        const Slots& w = s.b < 0 ? p.shared : p.own;
        const int64_t first = w.first(s.id, now.tile);
        const int rows = w.rows;
        const bool keep = r < nrow && !bars.failed;
        // O of a tile as [dh / 4][rows][4]: a warp's rows lie side by side
        float4* dst = reinterpret_cast<float4*>(w.o + first * DH) + half * (DH / 8) * rows + r;
#pragma unroll 1
        for (int c = 0; c < DH / 64; ++c) {
          uint32_t o[32];
          tmem_ld32(oc + 32 * c, o);
          tmem_wait_ld();
          if (keep) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(8 * c + e) * rows] =
                  make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
        if (half == 0 && r < nrow) *reinterpret_cast<float2*>(w.ml + (first + r) * 2) = bars.failed ? make_float2(NAN, NAN) : make_float2(m, l + l_other);
        tc_fence_before();
        mbar_arrive(&bars.o_free[t]);
        tile_sync();                                        // and the sums
        now = then;
      }
    } else if (warp == 16) {
      // -------------------------------------------------------- TMA: K0 V0 K1 V1 ..
      if (lane == 0) {
        // tile j of a segment's keys or values into the next ring entry
        auto fetch = [&](const Seg& s, int j, bool is_k) {
          const int y = static_cast<int>(tile_row(p, s, j)), slot = it % kSlots;
          if (bars.failed || (it >= kSlots && !wait(bars, &bars.empty[slot], ((it / kSlots) - 1) & 1, p.hdr, 620))) return;
          const CUtensorMap* map = s.b < 0 ? (is_k ? &map_ks : &map_vs) : (is_k ? &map_k : &map_v);
          const uint32_t dst = sbase + Sh::OFF_RING + slot * Sh::kTileB;
          mbar_expect_tx(&bars.full[slot], Sh::kTileB);
#pragma unroll
          for (uint32_t h = 0; h < Sh::kHalves; ++h) tma_load_2d(dst + h * Sh::kHalf, map, 64 * h, y, &bars.full[slot]);
          ++it;
        };
        // in the order of use below: a tile's keys ahead of the values of the tile before
        for (int i = 0; i < nseg && !bars.failed;) {
          const int n = group_of(p, bars.segs, i, nseg);
          int most = 0;
          for (int k = 0; k < n; ++k) {
            most = max(most, bars.segs[i + k].j1 - bars.segs[i + k].j0);
            fetch(bars.segs[i + k], bars.segs[i + k].j0, true);
          }
          for (int jj = 0; jj < most; ++jj)
            for (int k = 0; k < n; ++k) {
              const Seg& s = bars.segs[i + k];
              if (s.j0 + jj + 1 < s.j1) fetch(s, s.j0 + jj + 1, true);
              if (s.j0 + jj < s.j1) fetch(s, s.j0 + jj, false);
            }
          i += n;
        }
      }
      __syncwarp();
    } else if (warp == 17) {
      // -------------------------------------------------------- products: the whole warp waits, one lane issues
      const uint32_t lead = elect_one();
      constexpr uint32_t idS = idesc_bf16(false, kTile), idPV = idesc_bf16(true, DH);
      for (int i = 0; i < nseg;) {
        // of each row tile: its key tiles (0: it has no part), and whether it has its own
        const int n = __shfl_sync(0xffffffffu, group_of(p, bars.segs, i, nseg), 0);
        const Part part1 = part_of(p, bars.segs, i, n, 1);
        const int nj0 = __shfl_sync(0xffffffffu, bars.segs[i].j1 - bars.segs[i].j0, 0);
        const int nj1 = __shfl_sync(0xffffffffu, part1.seg < 0 ? 0 : bars.segs[part1.seg].j1 - bars.segs[part1.seg].j0, 0);
        const bool both = n == 1 && nj1 > 0;                // two row tiles of one segment: entries serve both
        uint32_t ek = 0, ev = 0;                            // ring entries of the keys and values in use
        auto scores = [&](int t) {
          if (t == 0 || !both) ek = it++;
          const uint32_t slot = ek % kSlots;
          wait(bars, &bars.full[slot], (ek / kSlots) & 1, p.hdr, 630);
          // the scores before, of whichever tile, are in registers
          if (last >= 0) {
            wait(bars, &bars.s_free[last], (ph_s >> last) & 1, p.hdr, 636);
            ph_s ^= 1u << last;
          }
          last = t;
          tc_fence_after();
          const uint64_t kd = sw128_desc(sbase + Sh::OFF_RING + slot * Sh::kTileB, 16, 1024);
          const uint64_t qd = sw128_desc(sbase + Sh::OFF_Q + t * Sh::kTileB, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks) {
            const uint32_t step = ((ks >> 2) * Sh::kHalf + (ks & 3) * 32) >> 4;      // addresses in 16 bytes; no carry: all below 2^18
            mma_bf16_warp(tmem + TM_S, qd + step, kd + step, idS, ks > 0 ? 1u : 0u, lead);
          }
          mma_commit_warp(&bars.s_full[t], lead);
          if (t == 1 || !both) mma_commit_warp(&bars.empty[slot], lead);
        };
        for (int t = 0; t < 2; ++t) {
          const int nj = t == 0 ? nj0 : nj1;
          if (nj == 0) continue;
          wait(bars, &bars.q_full[t], (ph_q >> t) & 1, p.hdr, 631);
          ph_q ^= 1u << t;
          scores(t);
        }
        const int most = max(nj0, nj1);
        for (int jj = 0; jj < most; ++jj) {
          for (int t = 0; t < 2; ++t) {
            const int nj = t == 0 ? nj0 : nj1;
            if (jj >= nj) continue;
            // the next scores first: they need nothing of this tile's softmax but its reading of the last ones
            if (jj + 1 < nj) scores(t);
            if (t == 0 || !both) {
              ev = it++;
              wait(bars, &bars.full[ev % kSlots], (ev / kSlots) & 1, p.hdr, 634);
              const Seg& s = bars.segs[t == 0 || both ? i : i + 1];
              const int r0 = s.len - (s.j0 + jj) * kTile;
              if (r0 < kTile) {
                // value rows behind the length: their weights are 0, and 0 times NaN would be NaN
                uint8_t* v = smem + Sh::OFF_RING + ev % kSlots * Sh::kTileB;
                for (int x = r0 * 8 + lane; x < kTile * 8; x += 32)
#pragma unroll
                  for (uint32_t h = 0; h < Sh::kHalves; ++h) *reinterpret_cast<uint4*>(v + h * Sh::kHalf + x * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
              }
            }
            const uint32_t slot = ev % kSlots;
            wait(bars, &bars.p_full[t], (ph_p >> t) & 1, p.hdr, 632);
            ph_p ^= 1u << t;
            if (jj == 0) {
              // O of the tile's last segment has been read
              if ((used >> t) & 1) {
                wait(bars, &bars.o_free[t], (ph_o >> t) & 1, p.hdr, 633);
                ph_o ^= 1u << t;
              }
              used |= 1u << t;
            }
            tc_fence_after();
            const uint64_t vd = sw128_desc(sbase + Sh::OFF_RING + slot * Sh::kTileB, Sh::kHalf, 1024);
            const uint32_t pa = tmem + TM_P + 64 * t;
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_bf16_ts_warp(tmem + TM_O + t * 128, pa + ks * 8, vd + ks * (16 * 128 >> 4), idPV, (jj > 0 || ks > 0) ? 1u : 0u, lead);
            mma_commit_warp(&bars.pv_done[t], lead);
            if (t == 1 || !both) mma_commit_warp(&bars.empty[slot], lead);
          }
        }
        i += n;
        if (__any_sync(0xffffffffu, bars.failed)) break;
      }
    }
    // segments and ring are free; the CTA goes on, or ends, as one
    gave_up = __syncthreads_or(bars.failed);
  }

  // copies in flight end before the CTA does, also after a wait that gave up
  if (warp == 16 && lane == 0)
    for (uint32_t e = it > kSlots ? it - kSlots : 0; e < it; ++e) wait_anyway(&bars.full[e % kSlots], (e / kSlots) & 1);
  if (warp == 17 && used != 0) {
    mma_commit_warp(&bars.last, elect_one());
    wait_anyway(&bars.last, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ------------------------------------------------------------------ parts, fp32
// The same runs and segments without tensor cores: 8 warps, four rows a warp at a time over tiles of 32
// keys in shared memory. Bound by shared memory: a product of the scores takes two words from there, each key
// is read again for each of a warp's rows, and four barriers stand between 32 keys and the next (8 sequences of
// 80 tokens, 32 heads, behind 4096 keys and up to 1500: 4340 us, 12 TFLOP/s). fp32 inputs are for small
// models and tests.
constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 4;               // of a warp
constexpr int kSimtKeys = 32;

template <int DH>
__global__ void __launch_bounds__(kSimtThreads) k_parts_simt(Params p) {
  constexpr int E = DH / 32;
  __shared__ float q_s[8 * kSimtRows][DH];
  __shared__ float kv_s[kSimtKeys][DH + 1];
  __shared__ Seg segs[kSegs];
  __shared__ int count, next;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t start = static_cast<int64_t>(blockIdx.x) * p.plan[kShare];
  const int units = p.plan[kUnits];
  int u = static_cast<int>(start < units ? start : units);
  const int u1 = static_cast<int>(start + p.plan[kShare] < units ? start + p.plan[kShare] : units);
  while (u < u1) {
    __syncthreads();
    if (tid == 0)
      next = describe(p, segs, &count, blockIdx.x, u, u1, p.unit0, p.ph0, p.tok_first, p.own_len, p.plan[kTokens], p.plan[kSharedLen],
                      p.plan[kSharedUnits]);
    __syncthreads();
    u = next;
    for (int i = 0; i < count; ++i) {
      const Seg s = segs[i];
      const bool apart = s.b < 0 && p.shared_table == nullptr;        // else in the caches' pages
      const float* kb = static_cast<const float*>(apart ? p.k_shared : p.k_cache);
      const float* vb = static_cast<const float*>(apart ? p.v_shared : p.v_cache);
      // the rows of both tiles one after another: row x is head x % G of token x / G
      const int rows = s.ntok * p.G;
      for (int x0 = 0; x0 < rows; x0 += 8 * kSimtRows) {
        __syncthreads();
        for (int e = tid; e < 8 * kSimtRows * DH; e += kSimtThreads) {
          const int x = x0 + e / DH;
          q_s[e / DH][e % DH] = x < rows ? static_cast<const float*>(p.q)[(static_cast<int64_t>(p.tok[s.tok0 + x / p.G]) * p.Hq + s.kvh * p.G + x % p.G) * DH + e % DH] *
                                               p.scale_log2
                                         : 0.f;
        }
        float m[kSimtRows], l[kSimtRows], o[kSimtRows][E], w[kSimtRows];
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) {
          m[r] = -INFINITY;
          l[r] = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] = 0.f;
        }
        for (int j = s.j0; j < s.j1; ++j) {
          const int64_t y = tile_row(p, s, j);
          const int keys = min(kTile, s.len - j * kTile);
          for (int k0 = 0; k0 < keys; k0 += kSimtKeys) {
            const int n = min(kSimtKeys, keys - k0);
            __syncthreads();
            for (int e = tid; e < kSimtKeys * DH; e += kSimtThreads) kv_s[e / DH][e % DH] = e / DH < n ? kb[(y + k0) * DH + e] : 0.f;
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kSimtRows; ++r) {
              const float* qr = q_s[warp * kSimtRows + r];
              float sc = 0.f;
#pragma unroll 8
              for (int e = 0; e < DH; ++e) sc = fmaf(qr[e], kv_s[lane][e], sc);
              sc = lane < n ? sc : -INFINITY;
              const float top = fmaxf(m[r], warp_max(sc));
              const float f = m[r] > -INFINITY ? exp2f(m[r] - top) : 0.f;
              w[r] = top > -INFINITY ? exp2f(sc - top) : 0.f;
              l[r] = l[r] * f + warp_sum(w[r]);
#pragma unroll
              for (int e = 0; e < E; ++e) o[r][e] *= f;
              m[r] = top;
            }
            __syncthreads();
            for (int e = tid; e < kSimtKeys * DH; e += kSimtThreads) kv_s[e / DH][e % DH] = e / DH < n ? vb[(y + k0) * DH + e] : 0.f;
            __syncthreads();
            for (int kk = 0; kk < n; ++kk) {
              float v[E];
#pragma unroll
              for (int e = 0; e < E; ++e) v[e] = kv_s[kk][lane + 32 * e];
#pragma unroll
              for (int r = 0; r < kSimtRows; ++r) {
                const float pk = __shfl_sync(0xffffffffu, w[r], kk);
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] = fmaf(pk, v[e], o[r][e]);
              }
            }
          }
        }
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) {
          const int x = x0 + warp * kSimtRows + r;
          if (x >= rows) continue;
          const int tk = x / p.G, tile = tk / p.tokens;
          const Slots& at = s.b < 0 ? p.shared : p.own;
          const int64_t first = at.first(s.id, tile);
          const int row = (tk - tile * p.tokens) * p.G + x % p.G;
          if (lane == 0) *reinterpret_cast<float2*>(at.ml + (first + row) * 2) = make_float2(m[r], l[r]);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int c = lane + 32 * e;
            at.o[first * DH + (c / 4 * at.rows + row) * 4 + c % 4] = o[r][e];
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ join
// four (dh 128) or two neighbours of a row
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 x = __ldg(reinterpret_cast<const float2*>(p + e));
      v[e] = x.x;
      v[e + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(p + e));
      v[e] = __uint_as_float(x << 16);
      v[e + 1] = __uint_as_float(x & 0xffff0000u);
    }
  }
}

// One warp for up to four heads of a token that share their keys: grid (tokens, groups of heads / 4). Lane i
// holds dims i N .. i N + N - 1 of each head; in a list of eight keys or segments it is also the one that
// has the score, maximum or weight of number i / 4 for head i % 4. The own block's keys are read here, one
// token after another: a key of another block or of an absent token is never touched, whatever it holds.
template <typename T, int DH>
__global__ void __launch_bounds__(128) k_join(Params p) {
  constexpr int N = DH / 32, H = 4, L = 8;
  // (Let in by k_parts once the plan is complete, to do the own block meanwhile, it made a call of two tokens
  // 34 us instead of 18.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, g_of = lane & 3, n_of = lane >> 2;
  const int i = blockIdx.x, groups = ceil_div(p.G, H), unit = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int all_tokens = __ldcg(p.plan + kTokens);
  if (i >= all_tokens || unit >= p.Hkv * groups) return;
  const int share = __ldcg(p.plan + kShare), shared_len = __ldcg(p.plan + kSharedLen), pair = 2 * p.tokens;
  const int token = __ldcg(p.tok + i), NT = p.NB * p.Dmax;
  const int b = token / NT, pos = (token - b * NT) % p.Dmax;
  const int own_first = __ldcg(p.tok_first + b), own_tokens = __ldcg(p.tok_first + b + 1) - own_first, own_u = __ldcg(p.plan + kSharedUnits) + __ldcg(p.unit0 + b), own_ph = __ldcg(p.ph0 + b), own_len = __ldcg(p.own_len + b);
  const int kvh = unit / groups, g0 = (unit - kvh * groups) * H, gn = min(H, p.G - g0);
  float q[H][N], o[H][N];
#pragma unroll
  for (int g = 0; g < H; ++g) {
    load_n<T, N>(static_cast<const T*>(p.q) + (static_cast<int64_t>(token) * p.Hq + kvh * p.G + g0 + min(g, gn - 1)) * DH + lane * N, q[g]);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      q[g][e] *= p.scale_log2;
      o[g][e] = 0.f;
    }
  }
  // of head g_of: reference maximum and sum so far
  float m = -INFINITY, l = 0.f;
  // takes in scores s with weights' factors a (of number n_of, head g_of); returns the weight
  auto take = [&](float s, float a) {
    float top = fmaxf(m, s);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float ref = top > -INFINITY ? top : 0.f;
    const float f = ex2_approx(m - ref), w = ex2_approx(s - ref);        // 0 for -inf, NaN where there is one
    float sum = a * w;
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    l = l * f + sum;
    m = top;
#pragma unroll
    for (int g = 0; g < H; ++g) {
      const float fg = __shfl_sync(0xffffffffu, f, g);
#pragma unroll
      for (int e = 0; e < N; ++e) o[g][e] *= fg;
    }
    return w;
  };

  // own block: slots k Dmax .. t
  const int64_t kv0 = ((static_cast<int64_t>(token) - pos) * p.Hkv + kvh) * DH + lane * N;
  const int64_t step = static_cast<int64_t>(p.Hkv) * DH;
  for (int c0 = 0; c0 <= pos; c0 += L) {
    float k[L][N], v[L][N], s[L * H];
#pragma unroll
    for (int c = 0; c < L; ++c) {
      const int64_t at = kv0 + min(c0 + c, pos) * step;      // behind the last one: that again, without weight
      load_n<T, N>(static_cast<const T*>(p.k_cand) + at, k[c]);
      load_n<T, N>(static_cast<const T*>(p.v_cand) + at, v[c]);
    }
#pragma unroll
    for (int c = 0; c < L; ++c)
#pragma unroll
      for (int g = 0; g < H; ++g) {
        s[c * H + g] = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) s[c * H + g] = fmaf(q[g][e], k[c][e], s[c * H + g]);
      }
    // 32 sums over 32 lanes, one to each lane: halves change hands
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int x = 0; x < d; ++x) {
        const bool up = lane & d;
        const float send = up ? s[x] : s[x + d];
        s[x] = (up ? s[x + d] : s[x]) + __shfl_xor_sync(0xffffffffu, send, d);
      }
    const bool there = c0 + n_of <= pos;
    const float w = take(there ? s[0] : -INFINITY, 1.f);
#pragma unroll
    for (int c = 0; c < L; ++c) {
      if (c0 + c > pos) break;
#pragma unroll
      for (int g = 0; g < H; ++g) {
        const float wg = __shfl_sync(0xffffffffu, w, c * H + g);
#pragma unroll
        for (int e = 0; e < N; ++e) o[g][e] = fmaf(wg, v[c][e], o[g][e]);
      }
    }
  }

  // the segments of a pair's units u_base + at kt .. + kt - 1
  auto join = [&](const Slots& part, int i0, int all, int u_base, int ph_base, int len) {
    if (len <= 0) return;
    const int kt = ceil_div(len, kTile), pr = i0 / pair, in = i0 - pr * pair, at = pr * p.Hkv + kvh;
    const int tile = in / p.tokens, row = (in - tile * p.tokens) * p.G + g0;
    const int w1 = tile_units(all, p.tokens), u = u_base + (at * (kt + kSetup) + kSetup) * w1, c0 = u / share, n = (u + (kt - 1) * w1) / share - c0 + 1;
    const int64_t id0 = static_cast<int64_t>(ph_base) + at + c0;
    for (int s0 = 0; s0 < n; s0 += L) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (s0 + n_of < n && g_of < gn) ml = __ldcg(reinterpret_cast<const float2*>(part.ml) + part.first(id0 + s0 + n_of, tile) + row + g_of);
      const float w = take(ml.x, ml.y);
      for (int c = 0; c < min(L, n - s0); c += 2) {
        float x[2][H][N];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          // (an odd last one twice, the second time without weight)
          const float* src = part.o + part.first(id0 + s0 + min(c + y, n - s0 - 1), tile) * DH + (lane * N / 4 * part.rows + row) * 4 + lane * N % 4;
#pragma unroll
          for (int g = 0; g < H; ++g)
#pragma unroll
            for (int e = 0; e < N; e += 2) {
              const float2 z = g < gn ? __ldcg(reinterpret_cast<const float2*>(src + 4 * g + e)) : make_float2(0.f, 0.f);
              x[y][g][e] = z.x;
              x[y][g][e + 1] = z.y;
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int g = 0; g < H; ++g) {
            const float wg = __shfl_sync(0xffffffffu, w, ((c + y) & (L - 1)) * H + g);
            if (c + y < n - s0) {
#pragma unroll
              for (int e = 0; e < N; ++e) o[g][e] = fmaf(wg, x[y][g][e], o[g][e]);
            }
          }
      }
    }
  };
  join(p.shared, i, all_tokens, 0, 0, shared_len);
  join(p.own, i - own_first, own_tokens, own_u, own_ph, own_len);

  const float inv = 1.f / l;
#pragma unroll
  for (int g = 0; g < H; ++g) {
    const float f = __shfl_sync(0xffffffffu, inv, g);
    if (g >= gn) continue;
    const int64_t at = (static_cast<int64_t>(token) * p.Hq + kvh * p.G + g0 + g) * DH + lane * N;
    if (sizeof(T) == 4 || p.out_f32) {
      float* out = static_cast<float*>(p.out) + at;
#pragma unroll
      for (int e = 0; e < N; e += 2) *reinterpret_cast<float2*>(out + e) = make_float2(o[g][e] * f, o[g][e + 1] * f);
    } else {
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
      for (int e = 0; e < N; e += 2) out[e / 2] = pack_bf16(o[g][e] * f, o[g][e + 1] * f);
    }
  }
}

// ------------------------------------------------------------------ host
// the most keys of the shared prompt and of a sequence, tokens of a pair, and pairs (x kv heads) of both
struct Extent {
  int64_t s_cap, p_cap, pair, ph_s, ph_o;
  explicit Extent(const ssd_attn_shared_args* a) {
    const int64_t NT = static_cast<int64_t>(a->NB) * a->Dmax;
    s_cap = a->shared_table != nullptr ? 128LL * a->shared_pages : a->S_max;
    p_cap = a->block_table != nullptr ? 128LL * a->pages_per_seq : a->P_max;
    pair = 2 * (kTile / (a->Hq / a->Hkv));
    ph_s = (a->B * NT + pair - 1) / pair * a->Hkv;
    ph_o = (NT + pair - 1) / pair * a->Hkv * a->B;
  }
  int64_t units() const { return 2 * (ph_s * ((s_cap + kTile - 1) / kTile + kSetup) + ph_o * ((p_cap + kTile - 1) / kTile + kSetup)); }
};

static int validate(const ssd_attn_shared_args* a) {
  if (a == nullptr) return SSD_ERR_INVALID;
  if (a->B < 0 || a->NB < 1 || a->Dmax < 1 || a->Hq < 1 || a->Hkv < 1 || a->P_max < 0) return SSD_ERR_INVALID;
  const bool apart = a->shared_table == nullptr;            // else k_shared, v_shared and S_max are not used
  if (apart && a->S_max < 0) return SSD_ERR_INVALID;
  if (a->dtype != SSD_F32 && a->dtype != SSD_BF16) return SSD_ERR_INVALID;
  if (a->out_dtype != a->dtype && a->out_dtype != SSD_F32) return SSD_ERR_INVALID;
  if (a->Hq % a->Hkv != 0 || !(a->scale >= 0.f)) return SSD_ERR_INVALID;
  if (a->dh != 64 && a->dh != 128) return SSD_ERR_UNSUPPORTED;
  if (a->Dmax > 256 || static_cast<int64_t>(a->NB) * a->Dmax > 8192 || a->Hq / a->Hkv > 64) return SSD_ERR_UNSUPPORTED;
  if (a->B > kMaxBatch || a->Hkv > 1024) return SSD_ERR_UNSUPPORTED;
  if (a->block_table != nullptr || a->shared_table != nullptr) {
    if (a->num_pages < 1) return SSD_ERR_INVALID;
    if (a->num_pages >= (1LL << 31) / 128 / a->Hkv) return SSD_ERR_UNSUPPORTED;
  }
  if (a->block_table != nullptr && a->pages_per_seq < 1) return SSD_ERR_INVALID;
  if (a->shared_table != nullptr && a->shared_pages < 1) return SSD_ERR_INVALID;
  // a shared prompt in pages lies in the pool of the sequences' pages
  if (a->shared_table != nullptr && a->block_table == nullptr) return SSD_ERR_INVALID;
  if (a->pages_per_seq > (1 << 20) || a->shared_pages > (1 << 20) || a->P_max > (1LL << 27) || (apart && a->S_max > (1LL << 27))) return SSD_ERR_UNSUPPORTED;
  if (a->block_table == nullptr && static_cast<double>(a->B) * a->Hkv * a->P_max >= 0x1p31) return SSD_ERR_UNSUPPORTED;
  if (apart && static_cast<double>(a->Hkv) * a->S_max >= 0x1p31) return SSD_ERR_UNSUPPORTED;
  if (a->B == 0) return SSD_OK;
  if (!a->q || !a->k_cand || !a->v_cand || !a->out || !a->shared_len || !a->prefix_len || !a->blk_len) return SSD_ERR_INVALID;
  if ((a->block_table != nullptr || a->P_max > 0) && (!a->k_cache || !a->v_cache)) return SSD_ERR_INVALID;
  if (apart && a->S_max > 0 && (!a->k_shared || !a->v_shared)) return SSD_ERR_INVALID;
  for (const void* x : {a->q, a->k_cache, a->v_cache, a->k_cand, a->v_cand, static_cast<const void*>(a->out)})
    if (!aligned(x, 16)) return SSD_ERR_UNSUPPORTED;
  if (apart && (!aligned(a->k_shared, 16) || !aligned(a->v_shared, 16))) return SSD_ERR_UNSUPPORTED;
  // units of work are counted in 32 bits
  if (Extent(a).units() >= (1LL << 30) || static_cast<int64_t>(a->B) * a->NB * a->Dmax * a->Hq >= (1LL << 31)) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

struct Layout {
  struct Part {
    size_t ml, o;
    int tiles, rows;
  };
  size_t plan, tok, tok_first, unit0, ph0, own_len, total;
  Part shared, own;
};

static int sm_count(int dev) {
  static std::once_flag once[kMaxDevices];
  static int n[kMaxDevices];
  std::call_once(once[dev], [dev] {
    if (cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n[dev] = 0;
  });
  return n[dev];
}

static int grid_of(const ssd_attn_shared_args* a, int sms) { return a->dtype == SSD_BF16 ? sms : 4 * sms; }

static Layout layout(const ssd_attn_shared_args* a, int ctas) {
  Layout L{};
  const int64_t NT = static_cast<int64_t>(a->NB) * a->Dmax, all = a->B * NT;
  const Extent x(a);
  size_t at = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = round_up(at + bytes, 256);
    return here;
  };
  L.plan = take(4 * kPlan);
  L.tok = take(4 * static_cast<size_t>(all));
  L.tok_first = take(4 * (static_cast<size_t>(a->B) + 1));
  L.unit0 = take(4 * (static_cast<size_t>(a->B) + 1));
  L.ph0 = take(4 * (static_cast<size_t>(a->B) + 1));
  L.own_len = take(4 * static_cast<size_t>(a->B));
  // every pair and head may be a segment, and every CTA but one may cut one more; its rows are those of `tokens` or, if
  // they are more than a row tile, of two row tiles
  auto part = [&](int64_t cap, int64_t ph, int64_t tokens) {
    const bool two = tokens > x.pair / 2;
    Layout::Part y = {0, 0, two ? 2 : 1, two ? kTile : static_cast<int>(tokens) * (a->Hq / a->Hkv)};
    const size_t rows = cap > 0 ? static_cast<size_t>(ph + ctas) * y.tiles * y.rows : 0;
    y.ml = take(rows * 8);
    y.o = take(rows * a->dh * 4);
    return y;
  };
  L.shared = part(x.s_cap, x.ph_s, all);
  L.own = part(x.p_cap, x.ph_o, NT);
  L.total = at;
  return L;
}

static bool kv_map(CUtensorMap* map, const void* base, uint64_t rows, int dh) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(dh), rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(dh) * 2};
  const cuuint32_t box[2] = {64, kTile};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH>
static int launch_parts(const Params& p, const ssd_attn_shared_args* a, cudaStream_t s) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  const int dev = current_device();
  std::call_once(once[dev], [dev] {
    err[dev] = cudaFuncSetAttribute(k_parts<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Shape<DH>::kSmem));
  });
  if (err[dev] != cudaSuccess) return SSD_ERR_CUDA;
  const uint64_t pool = static_cast<uint64_t>(a->num_pages) * a->Hkv * kTile;
  const uint64_t rs = a->shared_table != nullptr ? pool : static_cast<uint64_t>(a->Hkv) * a->S_max;
  const uint64_t ro = a->block_table != nullptr ? pool : static_cast<uint64_t>(a->B) * a->Hkv * a->P_max;
  const void* ks = a->shared_table != nullptr ? a->k_cache : a->k_shared;
  const void* vs = a->shared_table != nullptr ? a->v_cache : a->v_shared;
  // a part without keys gets no unit: its map only has to be a valid one
  CUtensorMap m[4];
  if (!kv_map(&m[0], rs > 0 ? ks : a->q, rs > 0 ? rs : 1, DH) || !kv_map(&m[1], rs > 0 ? vs : a->q, rs > 0 ? rs : 1, DH) ||
      !kv_map(&m[2], ro > 0 ? a->k_cache : a->q, ro > 0 ? ro : 1, DH) || !kv_map(&m[3], ro > 0 ? a->v_cache : a->q, ro > 0 ? ro : 1, DH))
    return SSD_ERR_CUDA;
  KernelTimer timer(SSD_KERNEL_ATTN_SHARED, s);
  if (launch_pdl(k_parts<DH>, dim3(static_cast<unsigned>(p.ctas)), dim3(kThreads), Shape<DH>::kSmem, s, m[0], m[1], m[2], m[3], p) != cudaSuccess)
    return SSD_ERR_CUDA;
  return SSD_OK;
}

template <typename T, int DH>
static cudaError_t launch_join(const Params& p, cudaStream_t s) {
  const int64_t tokens = static_cast<int64_t>(p.B) * p.NB * p.Dmax;
  const int units = p.Hkv * ceil_div(p.G, 4);
  return launch_pdl(k_join<T, DH>, dim3(static_cast<unsigned>(tokens), static_cast<unsigned>(ceil_div(units, 4))), dim3(128), 0, s, p);
}

}  // namespace shr
}  // namespace ssd

extern "C" size_t ssd_verify_attn_shared_workspace_size(const ssd_attn_shared_args* a) {
  using namespace ssd;
  if (shr::validate(a) != SSD_OK) return 0;
  const int dev = current_device();
  if (a->B == 0 || dev < 0) return sizeof(WsHeader);
  return shr::layout(a, shr::grid_of(a, shr::sm_count(dev))).total;
}

extern "C" int ssd_verify_attn_shared(const ssd_attn_shared_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssd;
  const int rc = shr::validate(a);
  if (rc != SSD_OK) return rc;
  if (a->B == 0) return SSD_OK;
  const int64_t es = a->dtype == SSD_BF16 ? 2 : 4, NT = static_cast<int64_t>(a->NB) * a->Dmax;
  const int64_t rows = a->B * NT * a->Hq * a->dh, cand = a->B * NT * a->Hkv * a->dh * es, row = static_cast<int64_t>(a->Hkv) * a->dh * es;
  const int64_t own = a->block_table != nullptr ? a->num_pages * 128 * row : a->B * a->P_max * row;
  const int64_t prompt = a->shared_table != nullptr ? 0 : a->S_max * row;
  const Span spans[] = {{a->out, rows * (a->out_dtype == SSD_F32 ? 4 : 2)}, {a->q, rows * es}, {a->k_shared, prompt}, {a->v_shared, prompt},
                        {a->k_cache, own}, {a->v_cache, own}, {a->k_cand, cand}, {a->v_cand, cand}, {a->shared_len, 4}, {a->prefix_len, 4LL * a->B},
                        {a->blk_len, 4LL * a->B * a->NB}, {a->shared_table, 4LL * a->shared_pages}, {a->block_table, 4LL * a->B * a->pages_per_seq}};
  if (overlap(spans, 1, 13)) return SSD_ERR_INVALID;
  const int dev = current_device();
  if (dev < 0) return SSD_ERR_CUDA;
  const int ctas = shr::grid_of(a, shr::sm_count(dev));
  if (ctas < 1) return SSD_ERR_CUDA;
  const shr::Layout L = shr::layout(a, ctas);
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < L.total) return SSD_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  shr::Params p = {};
  p.q = a->q;
  p.k_shared = a->k_shared;
  p.v_shared = a->v_shared;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.k_cand = a->k_cand;
  p.v_cand = a->v_cand;
  p.out = a->out;
  p.shared_len = a->shared_len;
  p.prefix_len = a->prefix_len;
  p.blk_len = a->blk_len;
  p.shared_table = a->shared_table;
  p.block_table = a->block_table;
  p.B = a->B;
  p.NB = a->NB;
  p.Dmax = a->Dmax;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.tokens = shr::kTile / p.G;
  p.S_max = a->S_max;
  p.P_max = a->P_max;
  p.num_pages = a->num_pages;
  p.shared_pages = a->shared_pages;
  p.pages_per_seq = a->pages_per_seq;
  p.scale_log2 = (a->scale != 0.f ? a->scale : 1.f / sqrtf(static_cast<float>(a->dh))) * kLog2e;
  p.out_f32 = a->out_dtype == SSD_F32;
  p.ctas = ctas;
  p.hdr = static_cast<WsHeader*>(ws);
  p.plan = reinterpret_cast<int32_t*>(w + L.plan);
  p.tok = reinterpret_cast<int32_t*>(w + L.tok);
  p.tok_first = reinterpret_cast<int32_t*>(w + L.tok_first);
  p.unit0 = reinterpret_cast<int32_t*>(w + L.unit0);
  p.ph0 = reinterpret_cast<int32_t*>(w + L.ph0);
  p.own_len = reinterpret_cast<int32_t*>(w + L.own_len);
  p.shared = {reinterpret_cast<float*>(w + L.shared.ml), reinterpret_cast<float*>(w + L.shared.o), L.shared.tiles, L.shared.rows};
  p.own = {reinterpret_cast<float*>(w + L.own.ml), reinterpret_cast<float*>(w + L.own.o), L.own.tiles, L.own.rows};
  if (launch_pdl(shr::k_plan, dim3(1), dim3(shr::kPlanThreads), 0, s, p) != cudaSuccess) return SSD_ERR_CUDA;
  if (a->dtype == SSD_BF16) {
    const int e = a->dh == 64 ? shr::launch_parts<64>(p, a, s) : shr::launch_parts<128>(p, a, s);
    if (e != SSD_OK) return e;
  } else {
    KernelTimer timer(SSD_KERNEL_ATTN_SHARED, s);
    const cudaError_t e = a->dh == 64 ? launch_pdl(shr::k_parts_simt<64>, dim3(ctas), dim3(shr::kSimtThreads), 0, s, p)
                                      : launch_pdl(shr::k_parts_simt<128>, dim3(ctas), dim3(shr::kSimtThreads), 0, s, p);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
  }
  cudaError_t e;
  if (a->dtype == SSD_BF16) e = a->dh == 64 ? shr::launch_join<uint16_t, 64>(p, s) : shr::launch_join<uint16_t, 128>(p, s);
  else e = a->dh == 64 ? shr::launch_join<float, 64>(p, s) : shr::launch_join<float, 128>(p, s);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  count_launch(3);
  return check_launch();
}
