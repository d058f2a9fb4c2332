// Attention over the 8-bit cache: argument checks, and the kernel for few packed rows
// (single tokens, short chains; any group size and head dim 64 or 128).
//
// Mathematics. With codes c, block scales sk and sv, and y_j = scale log2e (q.c_j) sk_j +
// log2 sv_j, the output is  sum_j 2^(y_j - M) c_j / sum_j 2^(y_j - M) / sv_j  for any M:
// the values' scale rides in the exponent, so no element is multiplied by it, and the
// denominator gets one multiplication by 1/sv for each group of keys of one block. M is
// the running maximum of y, moved only when it grows by more than 2^8; the weights of the
// output carry a factor 2^7 (at most 2^15 then), so that fp16 keeps the 11 bits of those down
// to 2^-21 of the largest: the tail of a long prefix beside one large key.
//
// What bounds it: the cache's bytes, read once (2 dh bytes a key and kv head). A warp
// takes two tiles of 16 keys a step and keeps its own running maximum, sum and output (online
// softmax), so warps share nothing until the end. Both products have the cache as their
// 16-row operand and the packed query rows as the 8-column one (S^T = K Q^T and
// O^T = V^T P^T, mma.sync), so eight rows, one token of most group sizes, waste
// nothing; a second column tile serves up to 16 rows. P^T turns from accumulator to operand
// by one movmatrix for 8 keys. Each warp has a
// ring of its own in shared memory, filled by one lane's tensor copies of 32 keys ahead of
// use, and no barrier with other warps. (The same loop with only its copies reads 6.8 TB/s;
// with 16-byte cp.async of each lane's own fragments 4.8.) Both products may permute an
// index, so fragments need no transpose: for K Q^T lane (g, t) holds elements
// 16t .. 16t+15 of each 64-element half of two keys, and Q is laid out alike; for
// V^T P^T it holds, for its four keys, the dh/8 output elements from dh/8 g on. K Q^T takes the
// codes as they are (e4m3 products, fp32 sums) against q as a sum of two e4m3 numbers; for
// V^T P^T they become fp16 exactly, by one conversion for two, against probabilities rounded
// to fp16 (at most 2^15): 11 bits where two e4m3 numbers would hold 8, for few instructions
// more. mma.sync is enough here: the matrix work is a fifth of the time the bytes take, and
// eight rows are a sixteenth of the smallest tcgen05 tile.
//
// Measured: 64 sequences of 2k-8k keys, 8 kv heads, one token each (672 MB): 105.4 us, 6.4 TB/s,
// 0.94 of a plain copy. One sequence of 4096 keys (8.4 MB): 8.7 us replayed from a graph, of which
// 1.2 are its bytes; launch, first loads, the own-block key and two merges are the rest.
//
// The CTAs of a cluster split the steps of a (sequence, kv head) evenly by its own length;
// rank 0 adds the own-block keys (bf16 products, probabilities as a sum of two bf16). Warps
// and then CTAs merge maxima, sums and outputs in a fixed order through shared memory.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "ssd_attn_quant.cuh"
#include "ssd_tc.cuh"

namespace ssd {

constexpr int kTileKeys = 16;             // rows of one product
constexpr int kStepKeys = 2 * kTileKeys;  // keys of a warp's step
constexpr int kMaxRanks = 16;             // CTAs of a cluster

// DH: head dim; N8: column tiles of eight packed rows; W: warps of a CTA; ST: steps in its
// rings; PER_SM: CTAs of an SM
template <int DH_, int N8_, int W_, int ST_, int PER_SM_>
struct RowsConfig {
  static constexpr int DH = DH_, N8 = N8_, W = W_, ST = ST_, PER_SM = PER_SM_;
  static constexpr int kThreads = W * 32;
  static constexpr int kTile = 8 * N8;                       // packed rows of a CTA
  static constexpr int kStep = 2 * kStepKeys * DH;           // K and V bytes of a step
  static constexpr int kWarpRing = ST * kStep;               // later the warp's output [row][DH] fp32
  static constexpr int kRing = W * kWarpRing;
  static constexpr int kScales = W * ST * 16;                // K scales of a step's tiles, V scales
  static constexpr int kBars = W * ST * 8 + 16;              // mbarriers, the failure flag, the sequence
  static constexpr int kStat = W * kTile * 8;                // maxima and sums of the warps
  static constexpr int kPeerStat = kMaxRanks * kTile * 8;    // ... of the cluster's CTAs
  static constexpr int kPeerOut = (kTile * DH + 4 * kMaxRanks) * 4;   // this CTA's share of their outputs
  static constexpr int OFF_SCALES = kRing, OFF_BARS = OFF_SCALES + kScales, OFF_STAT = OFF_BARS + kBars,
                       OFF_PEER_STAT = OFF_STAT + kStat, OFF_PEER_OUT = OFF_PEER_STAT + kPeerStat,
                       OFF_HERE = OFF_PEER_OUT + kPeerOut;
  static constexpr int kBytes = OFF_HERE + 16 + 1024;        // the base is aligned to 1024
  static_assert(kStep % 1024 == 0 && kTile * DH * 4 <= kWarpRing, "ring");
  static_assert(OFF_BARS % 16 == 0 && OFF_STAT % 16 == 0 && OFF_PEER_OUT % 16 == 0, "alignment");
};
constexpr unsigned long long kRowsWaitClocks = 1ull << 32;
constexpr float kRowsLag = 8.f, kRowsLift = 7.f, kRowsUnlift = 1.f / 128.f;   // log2, log2; sums carry no factor

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_b16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// an 8 x 8 matrix of 16-bit elements spread over the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 4 bytes of global memory to shared memory
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// over the eight lanes that hold one column of an accumulator
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Scores y (log2 units; -inf where masked) of keys g, g + 8 of U key tiles and rows 2t, 2t + 1
// of every column tile: moves the running maxima m, returns the factors on what was summed before and
// the references (with the factor 2^kRowsLift of the weights), and whether any lane of the warp needs
// the factors.
template <int N8, int U>
__device__ __forceinline__ bool move_max(float (&m)[N8][2], const float (&y)[U][N8][4], float (&ref)[N8][2],
                                         float (&alpha)[N8][2]) {
  bool moved = false;
#pragma unroll
  for (int n = 0; n < N8; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = fmaxf(y[0][n][i], y[0][n][2 + i]);
#pragma unroll
      for (int u = 1; u < U; ++u) top = fmaxf(top, fmaxf(y[u][n][i], y[u][n][2 + i]));
      top = column_max(top);
      alpha[n][i] = 1.f;
      if (top > m[n][i] + kRowsLag) {            // also the first keys: m is -inf
        alpha[n][i] = ex2_approx(m[n][i] - top);
        m[n][i] = top;
        moved = true;
      }
      ref[n][i] = m[n][i] == -INFINITY ? 0.f : m[n][i] - kRowsLift;
    }
  return __any_sync(0xffffffffu, moved);
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, C::PER_SM)
k_attn_quant_rows(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  AttnQuantParams p) {
  constexpr int DH = C::DH, N8 = C::N8, W = C::W, ST = C::ST, TILE = C::kTile;
  constexpr int KS = DH / 16;             // inner steps of K Q^T, and 16-element tiles of the output
  constexpr int EV = DH / 8;              // code bytes of a value row that a lane takes
  constexpr int KC = DH / 64;             // 16-byte chunks of a key row that a lane takes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* scales = reinterpret_cast<float4*>(smem + C::OFF_SCALES);  // [warp][stage]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BARS);
  volatile int* failed = reinterpret_cast<volatile int*>(bars + W * ST);
  volatile int* chosen = failed + 1;
  float2* stat = reinterpret_cast<float2*>(smem + C::OFF_STAT);            // [warp][row]: maximum, sum
  float2* peer_stat = reinterpret_cast<float2*>(smem + C::OFF_PEER_STAT);  // [rank][row]
  float4* peer_out = reinterpret_cast<float4*>(smem + C::OFF_PEER_OUT);    // [rank][share]
  uint8_t* present = smem + C::OFF_HERE;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t rank, S;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
  const int bk = blockIdx.x / S;
  int b = bk / p.Hkv;
  const int kvh = bk % p.Hkv;
  const int G = p.Hq / p.Hkv, NT = p.NB * p.Dmax;
  const int r0 = blockIdx.y * TILE, rows = min(TILE, NT * G - r0);

  if (tid == 0) {
    tc::prefetch_tmap(&map_k);
    tc::prefetch_tmap(&map_v);
    for (int i = 0; i < W * ST; ++i) tc::mbar_init(bars + i, 1);
    *failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // every CTA of the cluster runs before one writes to another's shared memory (waited for
  // before the merge)
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (p.longest_first) {
    // the CTAs of the longest prefixes start first, so that none of them is left for the end
    int* lens = reinterpret_cast<int*>(smem);
    const int mine = tid < p.B ? p.prefix_len[tid] : -1;
    lens[tid] = mine;
    tc::fence_async_smem();                          // tensor copies write the same place later
    __syncthreads();
    int before = 0;
    for (int i = 0; i < p.B; ++i) before += lens[i] > mine || (lens[i] == mine && i < tid) ? 1 : 0;
    if (tid < p.B && before == b) *chosen = tid;
    __syncthreads();
    b = *chosen;
  }
  int64_t P = p.prefix_len[b];
  // present rows of the tile; the CTAs of a cluster hold the same rows and leave together
  bool here = false;
  if (tid < rows) {
    const int tt = (r0 + tid) / G;
    here = tt % p.Dmax < p.blk_len[static_cast<int64_t>(b) * p.NB + tt / p.Dmax];
    present[tid] = here ? 1 : 0;
  }
  // rows of Q, and on rank 0 the first tile of own-block slots: loads that wait for nothing
  const int t_first = r0 / G, t_last = (r0 + rows - 1) / G;
  const int s_base = t_first / p.Dmax * p.Dmax;
  uint32_t raw[N8][KC * 2][4];
#pragma unroll
  for (int n = 0; n < N8; ++n) {
    const int row = n * 8 + g, rr = r0 + row;
    const bool ok = row < rows;
    const uint16_t* src = p.q + ((static_cast<int64_t>(b) * NT + (ok ? rr / G : 0)) * p.Hq + kvh * G + (ok ? rr % G : 0)) * DH + t4 * 16;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint4 x = ok ? *reinterpret_cast<const uint4*>(src + c * 64 + u * 8) : make_uint4(0u, 0u, 0u, 0u);
        raw[n][c * 2 + u][0] = x.x; raw[n][c * 2 + u][1] = x.y; raw[n][c * 2 + u][2] = x.z; raw[n][c * 2 + u][3] = x.w;
      }
  }
  const bool any_here = __syncthreads_or(here);
  if (!any_here) {
    if (S > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    return;
  }
  if (P < 0 || P > p.capacity) {
    if (tid == 0) record_error(p.hdr, SSD_ERR_DEVICE, 440);
    P = 0;
  }
  const int steps = static_cast<int>((P + kStepKeys - 1) / kStepKeys);
  const int step0 = static_cast<int>(static_cast<int64_t>(steps) * rank / S) + warp;
  const int step1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / S);

  // ---- the ring: step s into a stage, by one lane's tensor copies (K and V of 32 keys; rows
  // land swizzled) and four lanes' scales (an empty group past the end)
  auto page_of = [&](int s) -> int32_t {                // page of a step
    if (p.block_table == nullptr || s >= step1) return b;
    if (!in_range(s / (kPageTokens / kStepKeys), p.pages_per_seq, p.hdr, 445)) return 0;
    return p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + s / (kPageTokens / kStepKeys)];
  };
  uint8_t* my = smem + warp * C::kWarpRing;
  uint64_t* my_bar = bars + warp * ST;
  auto issue = [&](int s, int stage, int32_t page) {
    if (s < step1 && lane < 4) {
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) record_error(p.hdr, SSD_ERR_DEVICE, 441);
        page = 0;
      }
      // rows and blocks of the whole cache are counted in 31 bits
      const int place = p.block_table == nullptr ? s * kStepKeys : (s * kStepKeys) & (kPageTokens - 1);
      const int ph = page * p.Hkv + kvh;
      if (lane == 0) {
        const int row = ph * static_cast<int>(p.page_tokens) + place;
        const uint32_t dst = tc::smem_u32(my + stage * C::kStep);
        tc::mbar_expect_tx(my_bar + stage, C::kStep);
        tc::tma_load_2d(dst, &map_k, 0, row, my_bar + stage);
        tc::tma_load_2d(dst + kStepKeys * DH, &map_v, 0, row, my_bar + stage);
      }
      const int blocks = static_cast<int>(p.blocks);
      const int blk = min((place + (lane & 1) * kTileKeys) >> p.sb_log2, blocks - 1);
      if (in_range(static_cast<int64_t>(ph) * blocks + blk, p.num_pages * p.Hkv * blocks, p.hdr, 446))
        copy_async4(tc::smem_u32(scales + warp * ST + stage) + lane * 4,
                  (lane < 2 ? p.k_scale : p.v_scale) + static_cast<int64_t>(ph) * blocks + blk);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int32_t next_page = page_of(step0);
#pragma unroll
  for (int i = 0; i < ST; ++i) {
    issue(step0 + i * W, i, next_page);
    next_page = page_of(step0 + (i + 1) * W);
  }

  // ---- Q: lane (g, t) holds row g of every column tile. A power of two per row brings its
  // largest magnitude into [128, 256), and each element becomes the sum of two e4m3 numbers:
  // four significant bits and the four that a bf16 number has left, so exact down to 2^-9
  // of the row's largest and within 2^-17 of it below (half of e4m3's least step, 2^-10 of 128).
  uint32_t q[N8][KS / 4 * 2][4];                     // [8-byte group][words: first part, second part]
  float q_mul[N8][2];
#pragma unroll
  for (int n = 0; n < N8; ++n) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < KC * 2; ++k)
#pragma unroll
      for (int h = 0; h < 4; ++h) top = max(top, max((raw[n][k][h] << 16) & 0x7fff0000u, raw[n][k][h] & 0x7fff0000u));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // biased exponent of the factor 2^7 / 2^floor(log2 top); rows of zeros and subnormals, whose
    // factor would pass the largest exponent, take that, and infinities or NaN come out as NaN
    const int ex = static_cast<int>(top >> 23);
    const int up = min(254 + 7 - ex, 253);
    const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
#pragma unroll
    for (int k = 0; k < KC * 2; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {                  // four elements
        float x[4], y[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[2 * e] = __uint_as_float(raw[n][k][2 * h + e] << 16) * mul;
          x[2 * e + 1] = __uint_as_float(raw[n][k][2 * h + e] & 0xffff0000u) * mul;
        }
        if (ex == 255) x[0] = x[1] = x[2] = x[3] = __uint_as_float(0x7fffffffu);
        const uint32_t a = e4m3x2(x[0], x[1]), c = e4m3x2(x[2], x[3]);
        e4m3x2_to_f32(a, y[0], y[1]);
        e4m3x2_to_f32(c, y[2], y[3]);
        q[n][k][h] = a | c << 16;
        q[n][k][2 + h] = e4m3x2(x[0] - y[0], x[1] - y[1]) | e4m3x2(x[2] - y[2], x[3] - y[3]) << 16;
      }
    const float back = ex == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(254 - up) << 23) * p.scale_log2;
    // the accumulator's columns 2t, 2t + 1 are rows held by lanes (2t, .) and (2t + 1, .)
    q_mul[n][0] = __shfl_sync(0xffffffffu, back, t4 * 8);
    q_mul[n][1] = __shfl_sync(0xffffffffu, back, t4 * 8 + 4);
  }

  float m[N8][2], l[N8][2], o[N8][KS][4];
#pragma unroll
  for (int n = 0; n < N8; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
  }
  auto rescale = [&](const float (&alpha)[N8][2]) {
#pragma unroll
    for (int n = 0; n < N8; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          o[n][j][i] *= alpha[n][i];
          o[n][j][2 + i] *= alpha[n][i];
        }
        l[n][i] *= alpha[n][i];
      }
  };

  // ---- own-block keys (rank 0), one tile of 16 slots a step from the block of the tile's first row
  if (rank == 0) {
    const int lim = t_last + 1 - s_base;
    int tr[N8][2], lo[N8][2];                          // slot of a row and first slot of its block
#pragma unroll
    for (int n = 0; n < N8; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = n * 8 + 2 * t4 + i;
        tr[n][i] = r < rows ? (r0 + r) / G : -1;       // rows past the end see nothing
        lo[n][i] = r < rows ? tr[n][i] / p.Dmax * p.Dmax : 0;
      }
    for (int s = warp; s * kTileKeys < lim; s += W) {
      const int slot0 = s_base + s * kTileKeys;
      // values: lane's keys 2t, 2t + 1, 2t + 8, 2t + 9; elements g EV + ..
      uint32_t v[4][EV / 2];
      bool odd_value = false;                          // an infinity or NaN
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int slot = slot0 + 2 * t4 + (k & 1) + (k >> 1) * 8;
        const bool ok = slot <= t_last;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.v_cand + ((static_cast<int64_t>(b) * NT + (ok ? slot : t_last)) * p.Hkv + kvh) * DH + g * EV);
#pragma unroll
        for (int u = 0; u < EV / 8; ++u) {
          const uint4 x = ok ? src[u] : make_uint4(0u, 0u, 0u, 0u);
          v[k][4 * u] = x.x; v[k][4 * u + 1] = x.y; v[k][4 * u + 2] = x.z; v[k][4 * u + 3] = x.w;
        }
      }
      float c[N8][4] = {};
      // inner step k: elements 16 k + 4 t .. + 3 of a row
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint2 a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int slot = slot0 + h * 8 + g;
          a[h] = make_uint2(0u, 0u);
          if (slot <= t_last)
            a[h] = *reinterpret_cast<const uint2*>(p.k_cand + ((static_cast<int64_t>(b) * NT + slot) * p.Hkv + kvh) * DH +
                                                   k * 16 + t4 * 4);
        }
#pragma unroll
        for (int n = 0; n < N8; ++n) {
          uint2 v = make_uint2(0u, 0u);
          if (n * 8 + g < rows) {
            const int rr = r0 + n * 8 + g;
            v = *reinterpret_cast<const uint2*>(
                p.q + ((static_cast<int64_t>(b) * NT + rr / G) * p.Hq + kvh * G + rr % G) * DH + k * 16 + t4 * 4);
          }
          mma_b16(c[n], a[0].x, a[1].x, a[0].y, a[1].y, v.x, v.y);
        }
      }
      // scales of keys g and g + 8, from the largest finite magnitudes of their rows: each lane's own
      // 16 bits a key, two keys a word, then over the eight lanes of a key
      uint32_t top[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t most[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t x = 0;
#pragma unroll
          for (int u = 0; u < EV / 2; ++u) x = max_u16x2(x, v[2 * h + k][u] & 0x7fff7fffu);
          most[k] = max(x & 0xffffu, x >> 16);
          if (most[k] >= 0x7f80u) {
            odd_value = true;
            most[k] = 0;
#pragma unroll
            for (int u = 0; u < EV / 2; ++u) {
              const uint32_t a = v[2 * h + k][u] & 0x7fffu, b = v[2 * h + k][u] >> 16 & 0x7fffu;
              most[k] = max(most[k], max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
            }
          }
        }
        top[h] = most[0] | most[1] << 16;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top[h] = max_u16x2(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
      }
      odd_value = __any_sync(0xffffffffu, odd_value);
      float own_lv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        own_lv[h] = own_scale_log2(__shfl_sync(0xffffffffu, top[h], g >> 1) >> ((g & 1) * 16) & 0xffffu);
      float yy[1][N8][4], ref[N8][2], alpha[N8][2];
      float (&y)[N8][4] = yy[0];
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int slot = slot0 + (e >> 1) * 8 + g;
          c[n][e] = slot >= lo[n][e & 1] && slot <= tr[n][e & 1] ? c[n][e] * p.scale_log2 : -INFINITY;
          y[n][e] = c[n][e] + own_lv[e >> 1];
        }
      if (move_max<N8, 1>(m, yy, ref, alpha)) rescale(alpha);
#pragma unroll
      for (int n = 0; n < N8; ++n) {
        uint32_t hi[2], low[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w0 = ex2_approx(c[n][2 * h] - ref[n][0]), w1 = ex2_approx(c[n][2 * h + 1] - ref[n][1]);
          l[n][0] = fmaf(w0, kRowsUnlift, l[n][0]);
          l[n][1] = fmaf(w1, kRowsUnlift, l[n][1]);
          const uint32_t x = tc::pack_bf16(w0, w1);
          hi[h] = transpose8(x);
          low[h] = transpose8(tc::pack_bf16(w0 - __uint_as_float(x << 16), w1 - __uint_as_float(x & 0xffff0000u)));
        }
        if (!odd_value) {
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632),
                           a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
            mma_b16(o[n][j], a0, a1, a2, a3, hi[0], hi[1]);
            mma_b16(o[n][j], a0, a1, a2, a3, low[0], low[1]);
          }
        } else {
          // slots of other blocks and of absent tokens may hold anything, and 0 * inf is not
          // 0: key by key, for the rows that see it
#pragma unroll 1
          for (int k = 0; k < kTileKeys && slot0 + k <= t_last; ++k) {
            const uint16_t* src = p.v_cand + ((static_cast<int64_t>(b) * NT + slot0 + k) * p.Hkv + kvh) * DH + g * EV;
            const int from = (k & 7) * 4 + t4;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float ck = __shfl_sync(0xffffffffu, k < 8 ? c[n][i] : c[n][2 + i], from);
              if (slot0 + k < lo[n][i] || slot0 + k > tr[n][i]) continue;
              const float w = ex2_approx(ck - ref[n][i]);
#pragma unroll
              for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  o[n][j][2 * h + i] = fmaf(w, bf16_to_f32(src[2 * j + h]), o[n][j][2 * h + i]);
            }
          }
        }
      }
    }
  }

  // ---- prefix keys, two tiles a step. Which key of eight lane row g takes, and the order in
  // which lanes read their four value rows, keep the reads of the swizzled rows (16-byte chunk
  // c of row r lies at chunk c ^ (r & 7) for 128-byte rows, c ^ (r >> 1 & 3) for 64) free of
  // bank conflicts.
  const int kap = DH == 128 ? (g >> 1) | ((g & 1) << 2) : g;
  const int k_at = kap * DH + ((t4 ^ (DH == 128 ? kap : (kap >> 1) & 3)) << 4);
  const int swap = DH == 128 ? g & 1 : (g >> 1) & 1;
  int v_at[2];                                       // first and second key of four, as this lane reads them
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = DH == 128 ? t4 + 4 * (k ^ swap) : 2 * t4 + (k ^ swap);
    v_at[k] = r * DH + (DH == 128 ? (g ^ r) << 4 : (((g >> 1) ^ t4) << 4) + (g & 1) * 8);
  }
  const uint32_t sel[2] = {swap ? 0x1504u : 0x5140u, swap ? 0x3726u : 0x7362u};
  int stage = 0;
  uint32_t parity = 0;
  for (int s = step0; s < step1; s += W) {
    asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
    const bool arrived = mbar_wait_bounded(my_bar + stage, parity, failed, p.hdr, 442, kRowsWaitClocks);
    if (!__all_sync(0xffffffffu, arrived)) break;    // the warp leaves together
    __syncwarp();                                    // the scales are other lanes' copies
    uint8_t* st = my + stage * C::kStep;
    const float4 sc = scales[warp * ST + stage];
    const int left = static_cast<int>(P - static_cast<int64_t>(s) * kStepKeys);
    if (left < kStepKeys) {                          // codes past the prefix may be NaN: 0 * NaN is not 0
      for (int i = left * (DH / 16) + lane; i < kStepKeys * (DH / 16); i += 32)
        reinterpret_cast<uint4*>(st + kStepKeys * DH)[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
    }
    float c[2][N8][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[u][n][e] = 0.f;
#pragma unroll
      for (int ch = 0; ch < KC; ++ch) {
        const uint8_t* kt = st + u * kTileKeys * DH + (k_at ^ (ch * 64));
        const uint4 k0 = *reinterpret_cast<const uint4*>(kt), k1 = *reinterpret_cast<const uint4*>(kt + 8 * DH);
#pragma unroll
        for (int n = 0; n < N8; ++n)
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            mma_e4m3(c[u][n], k0.x, k1.x, k0.y, k1.y, q[n][ch * 2][2 * part], q[n][ch * 2][2 * part + 1]);
            mma_e4m3(c[u][n], k0.z, k1.z, k0.w, k1.w, q[n][ch * 2 + 1][2 * part], q[n][ch * 2 + 1][2 * part + 1]);
          }
      }
    }
    const float sk[2] = {sc.x, sc.y};
    const float lv[2] = {fmaxf(__log2f(sc.z), kLeastVScaleLog2), fmaxf(__log2f(sc.w), kLeastVScaleLog2)};
    float y[2][N8][4], ref[N8][2], alpha[N8][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[u][n][e] = fmaf(c[u][n][e], q_mul[n][e & 1] * sk[u], lv[u]);
    if (left < kStepKeys) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < N8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (u * kTileKeys + (e >> 1) * 8 + kap >= left) y[u][n][e] = -INFINITY;
    }
    if (move_max<N8, 2>(m, y, ref, alpha)) rescale(alpha);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float inv_sv = ex2_approx(-lv[u] - kRowsLift);     // and off with the factor
      uint32_t pb[N8][2];
#pragma unroll
      for (int n = 0; n < N8; ++n) {
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w0 = ex2_approx(y[u][n][2 * h] - ref[n][0]), w1 = ex2_approx(y[u][n][2 * h + 1] - ref[n][1]);
          sum[0] += w0;
          sum[1] += w1;
          pb[n][h] = transpose8(pack_f16(w0, w1));
        }
        l[n][0] = fmaf(sum[0], inv_sv, l[n][0]);
        l[n][1] = fmaf(sum[1], inv_sv, l[n][1]);
      }
      uint32_t v[4][EV / 4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* src = st + (kStepKeys + u * kTileKeys + (k >> 1) * 8) * DH + v_at[k & 1];
        if constexpr (EV == 16) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          v[k][0] = x.x; v[k][1] = x.y;
        }
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        // bytes 2j, 2j + 1 of two keys side by side: one pair of codes for each of two elements
        const uint32_t c0 = __byte_perm(v[0][j / 2], v[1][j / 2], sel[j & 1]), c1 = __byte_perm(v[2][j / 2], v[3][j / 2], sel[j & 1]);
        const uint32_t a0 = e4m3x2_to_f16x2(c0), a1 = e4m3x2_to_f16x2(c0 >> 16), a2 = e4m3x2_to_f16x2(c1),
                       a3 = e4m3x2_to_f16x2(c1 >> 16);
#pragma unroll
        for (int n = 0; n < N8; ++n) mma_f16(o[n][j], a0, a1, a2, a3, pb[n][0], pb[n][1]);
      }
    }
    __syncwarp();                                    // this stage has been read
    issue(s + ST * W, stage, next_page);
    next_page = page_of(s + (ST + 1) * W);
    if (++stage == ST) {
      stage = 0;
      parity ^= 1;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (*failed) {
    // a wait gave up: the copies still in flight write this CTA's shared memory, so give them
    // as long again before anything else does
    int one_more = 0;
    for (int i = 0; i < ST; ++i) mbar_wait_bounded(my_bar + i, i >= stage ? parity : parity ^ 1, &one_more, p.hdr, 443, kRowsWaitClocks);
  }

  // ---- merge the warps: each leaves its output in its own ring
#pragma unroll
  for (int n = 0; n < N8; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = n * 8 + 2 * t4 + i;
      float x = l[n][i];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (g == 0) stat[warp * TILE + r] = make_float2(m[n][i], x);
      if (r < rows) {
        float* dst = reinterpret_cast<float*>(my) + r * DH + g * EV;
#pragma unroll
        for (int j = 0; j < KS; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[n][j][i], o[n][j][2 + i], o[n][j + 1][i], o[n][j + 1][2 + i]);
      }
    }
  __syncthreads();
  // parts of a row are summed under their common maximum. A part without keys has maximum -inf, sum 0 and output 0; a NaN
  // score leaves the maximum and makes the sum NaN.
  const int quads = rows * (DH / 4), share = (quads + static_cast<int>(S) - 1) / static_cast<int>(S);
  auto store = [&](int e, float4 v, float L) {
    const int row = e / (DH / 4), rr = r0 + row, tt = rr / G;
    if (*failed || !present[row]) return;
    const int64_t at = ((static_cast<int64_t>(b) * NT + tt) * p.Hq + kvh * G + rr % G) * DH + e % (DH / 4) * 4;
    if (!in_range(at + 3, static_cast<int64_t>(p.B) * NT * p.Hq * DH, p.hdr, 447)) return;
    const float inv = __frcp_rn(L);
    v = make_float4(v.x * kRowsUnlift * inv, v.y * kRowsUnlift * inv, v.z * kRowsUnlift * inv, v.w * kRowsUnlift * inv);
    if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
  };
  auto add = [&](float4& v, float f, const float4& x) {
    v = make_float4(fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w));
  };
  if (S > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
  for (int e = tid; e < quads; e += C::kThreads) {
    const int row = e / (DH / 4);
    float2 st[W];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      st[w] = stat[w * TILE + row];
      M = fmaxf(M, st[w].x);
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = st[w].x == -INFINITY ? 1.f : ex2_approx(st[w].x - M);
      L = fmaf(f, st[w].y, L);
      add(v, f, reinterpret_cast<const float4*>(smem + w * C::kWarpRing)[e]);
    }
    if (S == 1) {
      store(e, v, L);
    } else {
      // to the CTA that owns this element, and the row's maximum and sum to every CTA
      const int to = e / share;
      const uint32_t dst = tc::map_peer(tc::smem_u32(peer_out + rank * share + (e - to * share)), to);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                   : "memory");
      const int c = e % (DH / 4);
      if (c < static_cast<int>(S)) {
        const uint32_t ds = tc::map_peer(tc::smem_u32(peer_stat + rank * TILE + row), c);
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(ds), "f"(M), "f"(L) : "memory");
      }
    }
  }
  if (S == 1) return;
  tc::cluster_sync();                                // from here on only this CTA's own memory is read
  for (int i = tid; i < share; i += C::kThreads) {
    const int e = static_cast<int>(rank) * share + i;
    if (e >= quads) break;
    const int row = e / (DH / 4);
    float M = -INFINITY, L = 0.f;
    for (uint32_t c = 0; c < S; ++c) M = fmaxf(M, peer_stat[c * TILE + row].x);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t c = 0; c < S; ++c) {
      const float2 st = peer_stat[c * TILE + row];
      const float f = st.x == -INFINITY ? 1.f : ex2_approx(st.x - M);
      L = fmaf(f, st.y, L);
      add(v, f, peer_out[c * share + i]);
    }
    store(e, v, L);
  }
}

// ------------------------------------------------------------------ host
static int validate(const ssd_attn_quant_args* a) {
  if (a == nullptr) return SSD_ERR_INVALID;
  if (a->B < 0 || a->NB < 1 || a->Dmax < 1 || a->Hq < 1 || a->Hkv < 1) return SSD_ERR_INVALID;
  if (a->out_dtype != SSD_BF16 && a->out_dtype != SSD_F32) return SSD_ERR_INVALID;
  if (a->Hq % a->Hkv != 0) return SSD_ERR_INVALID;
  if (!(a->scale >= 0.f) || isinf(a->scale)) return SSD_ERR_INVALID;
  if ((a->dh != 64 && a->dh != 128) || !scale_block_ok(a->scale_block)) return SSD_ERR_UNSUPPORTED;
  if (a->Dmax > 256 || static_cast<long long>(a->NB) * a->Dmax > 8192 || a->Hq / a->Hkv > 64) return SSD_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->B) * a->Hkv > (1 << 24)) return SSD_ERR_UNSUPPORTED;
  if (a->block_table != nullptr) {
    if (a->pages_per_seq < 1 || a->num_pages < 1) return SSD_ERR_INVALID;
    if (a->num_pages >= (1LL << 31) || a->num_pages * a->Hkv * kPageTokens >= (1LL << 31)) return SSD_ERR_UNSUPPORTED;
    if (a->pages_per_seq > (1 << 23)) return SSD_ERR_UNSUPPORTED;
  } else {
    if (a->P_max < 0) return SSD_ERR_INVALID;
    if (a->P_max > (1LL << 30) || static_cast<long long>(a->B) * a->Hkv * a->P_max >= (1LL << 31)) return SSD_ERR_UNSUPPORTED;
  }
  if (a->B == 0) return SSD_OK;
  if (!a->q || !a->k_cand || !a->v_cand || !a->out || !a->prefix_len || !a->blk_len) return SSD_ERR_INVALID;
  if ((a->block_table != nullptr || a->P_max > 0) && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale))
    return SSD_ERR_INVALID;
  if (!aligned(a->q, 16) || !aligned(a->k_cand, 16) || !aligned(a->v_cand, 16) || !aligned(a->out, 16) ||
      !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16))
    return SSD_ERR_UNSUPPORTED;
  const int64_t slots = static_cast<int64_t>(a->B) * a->NB * a->Dmax, rows = slots * a->Hq * a->dh, cand = 2 * slots * a->Hkv * a->dh;
  const bool paged = a->block_table != nullptr;
  const int64_t pages = paged ? a->num_pages : a->B, tokens = paged ? kPageTokens : a->P_max;
  const int64_t codes = pages * a->Hkv * tokens * a->dh;
  const int64_t scales = 4 * pages * a->Hkv * ((tokens + a->scale_block - 1) / a->scale_block);
  const Span spans[] = {{a->out, rows * (a->out_dtype == SSD_F32 ? 4 : 2)}, {a->q, 2 * rows}, {a->k_cand, cand},
                        {a->v_cand, cand}, {a->k_cache, codes}, {a->v_cache, codes}, {a->k_scale, scales},
                        {a->v_scale, scales}, {a->prefix_len, 4LL * a->B},
                        {a->blk_len, 4LL * a->B * a->NB}, {a->block_table, 4LL * a->B * a->pages_per_seq}};
  if (overlap(spans, 1, 11)) return SSD_ERR_INVALID;
  return SSD_OK;
}

// rows of dh codes, `box` of them a copy, swizzled over their whole length
static bool codes_map(CUtensorMap* map, const void* base, uint64_t rows, int dh, int box_rows) {
  tc::EncodeTiledFn enc = tc::encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(dh), rows > 0 ? rows : 1};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(dh)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(dh), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, dh == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Kernel attributes, once a device, and how many clusters of S CTAs are resident at once.
template <typename C>
static int rows_resident(int S) {
  static std::mutex mu;
  static bool ready[kMaxDevices];
  static int found[kMaxDevices][kMaxRanks + 1];
  const int dev = current_device();
  if (dev < 0) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(k_attn_quant_rows<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes) != cudaSuccess ||
        cudaFuncSetAttribute(k_attn_quant_rows<C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    for (int n = 1; n <= kMaxRanks; ++n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(n), 1, 1);
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::kBytes;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(n);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int count = 0;
      if (cudaOccupancyMaxActiveClusters(&count, k_attn_quant_rows<C>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        count = 0;
      }
      found[dev][n] = count;
    }
    ready[dev] = true;
  }
  return found[dev][S];
}

// CTAs that split a sequence, at most `most`: those whose waves of resident clusters cost least. A CTA
// takes its share of the longest sequence's steps and a few beside them. A sequence or two (`even`)
// leave nothing short for a second wave, which then costs as much as the first (one sequence
// of 32768 keys: 20.1 us by 12 CTAs, 31.3 by 16, of which one cluster of eight waits). Of many the
// host knows only the capacity: where the lengths are equal waves count in full, where they vary
// (the longest started first) they run into each other, so the mean of both is taken; a fuller GPU
// makes each CTA slower, the more the less it computes a byte. Replayed from a graph, flushed, one
// token and 8 kv heads, us by 1 .. 6 CTAs: 16 sequences of 4096 56.7 43.5 39.9 *41.3 52.5 50.3, 32 68.7
// *66.7 77.3 70.0 78.9 74.1, of 2k-8k 111.6 85.8 82.7 *79.0 86.6 85.1, 64 152.2 *130.6 135.8 137.1
// 141.9 149.3 (* the one taken); 32 rows of 4 sequences of 4096 58.5 38.1 35.9 *30.9 49.7 46.6.
template <typename C>
static int rows_split(long long groups, long long keys, int most, bool even) {
  const double iters = static_cast<double>(std::max<long long>(1, (keys + C::W * kStepKeys - 1) / (C::W * kStepKeys)));
  const double slower = C::N8 == 1 ? 0.75 : 0.25;
  int best = 0;
  double cost = 0;
  for (int S = 1; S <= most && S <= iters; ++S) {
    const int clusters = rows_resident<C>(S);
    if (clusters <= 0) continue;
    const double waves = static_cast<double>(groups) / clusters;
    const double c = even ? (iters / S + 6.) * std::ceil(waves)
                          : (iters / S + 8.) * ((std::ceil(waves) + std::max(waves, 1.)) / 2 + slower * std::min(waves, 1.));
    if (best == 0 || c < (even ? 1. : 0.98) * cost) {
      cost = c;
      best = S;
    }
  }
  return best;
}

template <typename C>
static int rows_launch(const AttnQuantParams& p, int rows, int S, cudaStream_t s) {
  if (S < 1 || rows_resident<C>(S) <= 0) return SSD_ERR_CUDA;
  const uint64_t cache_rows = static_cast<uint64_t>(p.num_pages) * p.Hkv * p.page_tokens;
  CUtensorMap map_k, map_v;
  // an empty cache is never read, but a map needs an address and a row
  const void *kb = cache_rows > 0 ? p.k_cache : static_cast<const void*>(p.q), *vb = cache_rows > 0 ? p.v_cache : kb;
  if (!codes_map(&map_k, kb, cache_rows, C::DH, kStepKeys) || !codes_map(&map_v, vb, cache_rows, C::DH, kStepKeys))
    return SSD_ERR_CUDA;
  AttnQuantParams q = p;
  q.longest_first = p.B > 1 && p.B <= C::kThreads ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.B) * p.Hkv * S),
                     static_cast<unsigned>((rows + C::kTile - 1) / C::kTile), 1);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, k_attn_quant_rows<C>, map_k, map_v, q) != cudaSuccess) {
    cudaGetLastError();
    return SSD_ERR_CUDA;
  }
  count_launch();
  return check_launch();
}

template <int DH, int N8>
static int rows_choose(const AttnQuantParams& p, int rows, cudaStream_t s) {
  // Few sequences: latency counts, so eight warps and up to 16 CTAs share each (a token over
  // 4096 keys of 8 kv heads: 8.6 us, with the other shape 11.0). Many: four small CTAs of an SM
  // keep it reading while one starts or ends (64 sequences of 2k-8k: 107 us; three of four
  // warps 119, six of two 120, one of eight 123). Sixteen rows need the registers of eight
  // warps an SM: two CTAs of four (32 sequences of 1000 keys 31.9 us, one of eight 44.6; 64 of
  // 2k-8k now 163).
  using Few = RowsConfig<DH, N8, 8, 3, 1>;
  using Many = std::conditional_t<N8 == 1, RowsConfig<DH, N8, 3, 2, 4>, RowsConfig<DH, N8, 4, 2, 2>>;
  const long long groups = static_cast<long long>(p.B) * p.Hkv * ((rows + 8 * N8 - 1) / (8 * N8));
  if (groups * 8 <= 152) return rows_launch<Few>(p, rows, rows_split<Few>(groups, p.capacity, kMaxRanks, true), s);
  return rows_launch<Many>(p, rows, rows_split<Many>(groups, p.capacity, kMaxRanks, false), s);
}

}  // namespace ssd

extern "C" size_t ssd_verify_attn_quant_workspace_size(const ssd_attn_quant_args* a) {
  return ssd::validate(a) == SSD_OK ? sizeof(ssd::WsHeader) : 0;
}

extern "C" int ssd_verify_attn_quant(const ssd_attn_quant_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssd;
  const int st = validate(a);
  if (st != SSD_OK) return st;
  if (a->B == 0) return SSD_OK;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
  AttnQuantParams p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k_cache = static_cast<const uint8_t*>(a->k_cache);
  p.v_cache = static_cast<const uint8_t*>(a->v_cache);
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.k_cand = static_cast<const uint16_t*>(a->k_cand);
  p.v_cand = static_cast<const uint16_t*>(a->v_cand);
  p.out = a->out;
  p.prefix_len = a->prefix_len;
  p.blk_len = a->blk_len;
  p.block_table = a->block_table;
  p.B = a->B; p.NB = a->NB; p.Dmax = a->Dmax; p.Hq = a->Hq; p.Hkv = a->Hkv;
  p.pages_per_seq = a->pages_per_seq;
  p.sb_log2 = log2_of(a->scale_block);
  p.out_f32 = a->out_dtype == SSD_F32 ? 1 : 0;
  const float scale = a->scale != 0.f ? a->scale : 1.f / sqrtf(static_cast<float>(a->dh));
  p.scale_log2 = scale * kLog2e;
  const bool paged = a->block_table != nullptr;
  p.capacity = paged ? static_cast<int64_t>(a->pages_per_seq) * kPageTokens : a->P_max;
  p.page_tokens = paged ? kPageTokens : a->P_max;
  p.num_pages = paged ? a->num_pages : a->B;
  p.blocks = (p.page_tokens + a->scale_block - 1) / a->scale_block;
  p.hdr = static_cast<WsHeader*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rows = a->NB * a->Dmax * (a->Hq / a->Hkv);
  KernelTimer timer(SSD_KERNEL_VERIFY_ATTN, s);
  // Beyond 16 rows this kernel reads the cache once for each 16; the tensor-core kernel costs the
  // same up to 128 but starts and merges more slowly. So this one up to 48 rows while its CTAs run
  // at once and have little to read. Replayed from a graph, cold, us by this and by the other: 20 rows of
  // 4 sequences of 1024 keys, 8 kv heads, 19.6 and 21.6 (head dim 64: 15.5 and 19.6), one of 4096
  // with 2 kv heads 17.5 and 23.7 (15.5 and 19.6); at or past the limits, 16 sequences of 500 21.6
  // and 21.6 (17.5 and 19.6), 4 of 16384 71 and 54 (52 and 50), 48 rows of 8192 28 and 26 (22 and 24).
  const long long groups = static_cast<long long>(p.B) * p.Hkv * ((rows + 15) / 16);
  const bool small = rows <= 16 || (rows <= 48 && groups <= 152 && groups * p.capacity <= (1 << 17));
  if (!small && attn_quant_tc_applies(p)) return attn_quant_tc_launch(p, a->dh, s);
  // eight rows or sixteen in a CTA
  if (a->dh == 128) return rows <= 8 ? rows_choose<128, 1>(p, rows, s) : rows_choose<128, 2>(p, rows, s);
  return rows <= 8 ? rows_choose<64, 1>(p, rows, s) : rows_choose<64, 2>(p, rows, s);
}
