// Attention over the 8-bit cache for many packed rows on the tensor cores (tcgen05): a verification of many candidate tokens. The mathematics is that of
// ssd_attn_quant.cu; what differs is who does the products.
//
// Precision on 8-bit operands. The codes go into the products as they lie in the cache
// (kind::f8f6f4, fp32 sums). Q and P, which have more bits, are sums of two and three 8-bit numbers, one
// product each into the same accumulator. q (8 significant bits) is two e4m3 numbers, exact but
// for what lies under 2^-17 of its row's largest element. A probability, rounded to fp16, is the sum
// of three e5m2 numbers, each the rest of the ones before: three times three bits and two signs,
// exact. e5m2's range lets the largest lie at 2^11 to 2^15, so that all 11 bits are there down to 2^-17
// of the largest, nine at 2^-19, and smaller ones are off by at most 2^-28 of it. A long prefix needs
// that: beside one key of a large weight (or a block of a large value scale) its tail is 2^-15 each and
// most of the mass together. With an e4m3 and an e5m2 number, 8 bits down to 2^-10 and three at 2^-15,
// such a tail of 32768 keys was 1.3% off; the third product takes 2% more time in a single call, 8% in
// a loop that the GPU's power limits (4 sequences of 32768 keys), 6% in the serving batch. No code is converted.
// (Converting each tile to fp16 in shared memory would move 64 KB more per tile through it.)
//
// Rows. The G query heads of the present tokens pack into rows (absent tokens take none, so a
// batch with few present candidates runs few row tiles); a CTA owns 128 of them and one share
// of the prefix, the S CTAs of a row tile form a cluster, rank 0 also takes the own-block keys
// (bf16, masked), and the shares are merged on chip.
//
// Per CTA (384 threads, one CTA per SM, all 512 TMEM columns):
//   warps 0-3, 8-11  two threads per row, 64 columns of a tile each (one warp a scheduler left
//              it waiting on its own latencies: 1.7 us a tile): Q into shared memory (two e4m3
//              parts, swizzled; rank 0 also bf16), then the online softmax of each 128-key tile,
//              read from TMEM once: per 16 keys one K factor, one log2 of the V factor and one
//              weight 1/sv of the sum. A barrier of the two warps that share rows tells whether one of their
//              references has to move, which is rare. P goes back to TMEM over the tile's S
//              buffer (three parts of 32 columns, four keys a word; bf16 pairs for own-block
//              tiles). In fp16 the parts are the upper bytes of a probability's bits and of what
//              is left, so no format conversion is needed. On rank 0 they also take infinities and NaN
//              out of own-block values;
//   warp 4     TMEM allocation, then the producer of the K tiles;
//   warp 6     the producer of the V tiles; it clears the value rows past the prefix (codes
//              there may be NaN, and 0 * NaN is not 0);
//   warp 5     issues S = Q K^T, up to three tiles ahead of the softmax;
//   warp 7     issues O += P V (two issuing threads, so that neither's waits hold the other back).
// Head dim 64: the same layouts, with zeros behind a row's 64 codes (filled in by the tensor copies),
// half the products of S and half of O's columns kept: 320 rows of one sequence of 4096 keys 23.7 us
// where the kernel for few rows takes 48.3, of 32 of 2048 161 and 446.
// Shared memory: Q (64 KB), then four 16 KB slots each for K and V. A prefix tile takes one
// slot of each, an own-block tile (bf16) two.
// TMEM columns: S buffers 0-127, 128-255, 256-383, O 384-511.
// The merge is that of ssd_attn_tc.cu: rows as 16-bit integers with a power-of-two scale per
// DH / 2 columns, one bulk copy to each CTA that owns rows.
//
// What bounds it, and what it measured: a 128 x 128 tile takes 2020 to 2270 clocks on 8 to 64 SMs and
// 2300 on all, where its 20 instructions of products need 1280 at the tensor pipe's best: the
// softmax beside them. (With two products of P V, 16 instructions, it was 2050 and 2300. Measured
// then, four sequences of 32768 keys, us: four threads a row 470 where this took 464, turns of
// two softmax groups on alternate tiles 509, a second accumulator for them 570, a single thread a
// row 624.) Four sequences of 32768 keys and 800 rows: 468 us for a single call, 490-500 in a loop
// (0.87 PFLOP/s counted as bf16), where all SMs busy for long take the GPU to its power limit: a loop of
// 152 CTAs drew 1355 W with the power cap active and the clock at 1762 of 2070 MHz, on 64 SMs 805 W at
// 2070. 32 sequences of 1k-16k, nine blocks of 16, some absent: 285-329 us between draws. One of 4096
// keys, 320 rows: 21 us, Q's conversion, an own-block tile, seven tiles and the merge in a row.
// Waits are bounded; on expiry the CTA records SSD_ERR_TIMEOUT, skips what is left, gives its own
// copies and products in flight as long again, and exits through the cluster barriers.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "ssd_attn_quant.cuh"
#include "ssd_tc.cuh"

namespace ssd {
namespace qtc {

using namespace tc;

constexpr int BM = 128;                   // packed rows per CTA
constexpr int BN = 128;                   // keys per tile
constexpr int SLOTS = 4;                  // ring slots of K, and of V
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int SBUF = 3;
constexpr uint32_t TM_S = 0, TM_O = SBUF * BN;
constexpr uint32_t PART = BN / 4;         // columns of one part of the probabilities
constexpr uint32_t kSlot = 16384;         // 128 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t OFF_Q8 = 0;            // two parts
constexpr uint32_t OFF_QB = 2 * kSlot;    // bf16, two 64-column halves
constexpr uint32_t OFF_K = 4 * kSlot;
constexpr uint32_t OFF_V = OFF_K + SLOTS * kSlot;
constexpr uint32_t OFF_BAR = OFF_V + SLOTS * kSlot;
constexpr uint32_t kBarBytes = 5120;
constexpr uint32_t kSmemBytes = OFF_BAR + kBarBytes + 1024;   // + slack to align the base to 1024
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
constexpr unsigned long long kWaitClocks = 1ull << 32;
constexpr int kMaxSplit = 16;
constexpr int kSoftmax = 256;             // softmax threads
constexpr int FACTORS = 8;                // prefix tiles whose factors are kept
constexpr int kMaxBlocks = 8192;          // NB: the block ends are kept in the ring at first
static_assert((2 * BM + kMaxSplit) * (2 * 128 + 16) <= static_cast<int>(2 * SLOTS * kSlot), "merge buffers fit in the ring");
static_assert(kMaxBlocks * 4 <= static_cast<int>(2 * SLOTS * kSlot), "block ends fit in the ring");

struct Bars {
  uint64_t full_k[SLOTS], full_v[SLOTS], empty_k[SLOTS], empty_v[SLOTS];
  uint64_t q_full;
  // s_free: P V of the tile in the buffer is done. Also what a rescaling of O waits for: S of tile j - 1
  // was issued behind the phase of tile j - 4, so a wait for tile j - 1's cannot take an earlier one.
  uint64_t s_full[SBUF], p_full[SBUF], s_free[SBUF];
  uint64_t o_done;                        // every product into O is done
  uint64_t v_clean;                       // the value rows past the prefix are zeros
  // an own-block tile's values are finite. One barrier a ring slot: an arrival for tile j + 4
  // follows the copy into the slots that P V of tile j left, whose issue waited for tile j's phase,
  // so no phase passes the wait for the one before.
  uint64_t own_clean[SLOTS];
  uint64_t recv_full;
  uint64_t drained[2];                    // after a wait gave up: the products issued so far are done
  uint32_t tmem_base;
  int failed;
  int sent[2];                            // ring units that the K and V producers have copied
  int odd_own;                            // an own-block value was not finite
  int seq, rows;                          // the sequence; its present rows
  int row_slot[BM];                       // candidate slot of a row of this tile
  int row_at[BM];                         // its place in the sequence's Q and output, in rows of DH
  float pair[2][BM];                      // a value of each half of a row
  alignas(16) float own_lv[2][BN];                    // log2 of the scales of an own-block tile's value rows, in turns
  // of a prefix tile's eight groups of 16 keys: K factor, log2 of the V factor, 1 / V factor
  float4 factors[FACTORS][3][2];
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

__device__ __forceinline__ bool mbar_wait(Bars& bars, uint64_t* bar, uint32_t parity, WsHeader* hdr, int where) {
  return mbar_wait_bounded(bar, parity, &bars.failed, hdr, where, kWaitClocks);
}

// instruction descriptor, kind::f8f6f4: A e4m3 (or e5m2), B e4m3, fp32 D, M = 128, N = n
__host__ __device__ constexpr uint32_t idesc_f8(bool a_e5m2, bool b_mn_major, uint32_t n) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_mn_major ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// A in TMEM: M rows on the lanes, four K elements a column
__device__ __forceinline__ void mma_f8_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// merged rows travel as 16-bit integers, two a word
__device__ __forceinline__ uint32_t pack_i16(float x0, float x1, float s) {
  const uint32_t a = __float_as_uint(fmaf(x0, s, 12582912.f)), b = __float_as_uint(fmaf(x1, s, 12582912.f));
  return __byte_perm(a, b, 0x5410);
}
__device__ __forceinline__ float2 unpack_i16(uint32_t w) {
  const uint32_t f = w ^ 0x80008000u;
  return make_float2(__uint_as_float(__byte_perm(f, 0x4B000000u, 0x7610)) - 8421376.f,
                     __uint_as_float(__byte_perm(f, 0x4B000000u, 0x7632)) - 8421376.f);
}

// ------------------------------------------------------------------ softmax pieces
// Probabilities carry a factor 2^11 against their reference and may grow by another 2^4 before
// the reference moves: at most 2^15, under e5m2's 57344. Sums carry no factor.
constexpr float kLift = 11.f, kLag = 4.f, kUnlift = 1.f / 2048.f;

// the factors of four groups of 16 keys (64 columns)
struct Groups {
  float k[4];      // score to log2 units
  float lv[4];     // log2 of the V factor
  float w[4];      // weight of the group's sum: 1 / V factor
};

__device__ __forceinline__ void load64(uint32_t taddr, uint32_t* v) {
  tmem_ld32(taddr, v);
  tmem_ld32(taddr + 32, v + 32);
  tmem_wait_ld();
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// two fp32 operations in one instruction
__device__ __forceinline__ void fma2(float& x, float& y, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(x), "=f"(y) : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a0, float a1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y) : "f"(a0), "f"(a1));
}

// own-block tile: largest y of the columns [lo, hi) of 64, whose keys have a scale each
__device__ __forceinline__ float own_max(const uint32_t (&v)[64], float k, const float* lv, int lo, int hi) {
  float top = -INFINITY;
#pragma unroll
  for (int c = 0; c < 64; c += 4) {
    const float4 f = *reinterpret_cast<const float4*>(lv + c);
    const float l[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e >= lo && c + e < hi) top = fmaxf(top, fmaf(__uint_as_float(v[c + e]), k, l[e]));
  }
  return top;
}

// largest y of the columns below hi of 64 (MASK), or of all
template <bool MASK>
__device__ __forceinline__ float chunk_max(const uint32_t (&v)[64], const Groups& f, int hi) {
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int c = 16 * q; c < 16 * q + 16; c += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = !MASK || c + e < hi ? __uint_as_float(v[c + e]) : -INFINITY;
      a = max3(a, x[0], x[1]);
      b = max3(b, x[2], x[3]);
    }
    a = fmaxf(a, b);
    if (!MASK || a > -INFINITY) top = fmaxf(top, fmaf(a, f.k[q], f.lv[q]));   // an empty group's factors may be anything
  }
  return top;
}

// prefix tile: 2^(y - ref + lift) as three e5m2 parts, four keys a word, at paddr, paddr + PART and
// paddr + 2 PART; returns the sum weighted by 1 / V factor
template <bool MASK>
__device__ __forceinline__ float chunk_parts(const uint32_t (&v)[64], uint32_t paddr, const Groups& f, int hi, float ref) {
  uint32_t p1[16], p2[16], p3[16];
  float total = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // fp16 bits are, from bit 8 up, those of the e5m2 number: half of bit 8 rounds, and what a part
    // leaves is exact in fp16
    const float off = f.lv[q] - ref + kLift;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int c = 16 * q; c < 16 * q + 16; c += 4) {
      uint32_t t1[2], t2[2], t3[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x, y;
        fma2(x, y, __uint_as_float(v[c + 2 * h]), __uint_as_float(v[c + 2 * h + 1]), f.k[q], off);
        x = ex2_approx(x);
        y = ex2_approx(y);
        if (MASK) {
          if (c + 2 * h >= hi) x = 0.f;
          if (c + 2 * h + 1 >= hi) y = 0.f;
        }
        add2(s0, s1, x, y);
        uint32_t w, left;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
        t1[h] = w + 0x00800080u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(left) : "r"(w), "r"(t1[h] & 0xff00ff00u));
        t2[h] = left + 0x00800080u;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(left) : "r"(left), "r"(t2[h] & 0xff00ff00u));
        t3[h] = left + 0x00800080u;
      }
      p1[c / 4] = __byte_perm(t1[0], t1[1], 0x7531);
      p2[c / 4] = __byte_perm(t2[0], t2[1], 0x7531);
      p3[c / 4] = __byte_perm(t3[0], t3[1], 0x7531);
    }
    const float s = s0 + s1;
    if (!MASK || 16 * q < hi) total = fmaf(s, f.w[q], total);
  }
  tmem_st16(paddr, p1);
  tmem_st16(paddr + PART, p2);
  tmem_st16(paddr + 2 * PART, p3);
  return total * kUnlift;
}

// own-block tile: 2^(y - ref + lift) as bf16 pairs over the columns [lo, hi); returns the sum
// of the rounded values
__device__ __forceinline__ float chunk_pairs(const uint32_t (&v)[64], uint32_t paddr, float k, int lo, int hi, float ref) {
  uint32_t pk[32];
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    float x = ex2_approx(fmaf(__uint_as_float(v[c]), k, kLift - ref)), y = ex2_approx(fmaf(__uint_as_float(v[c + 1]), k, kLift - ref));
    if (c < lo || c >= hi) x = 0.f;
    if (c + 1 < lo || c + 1 >= hi) y = 0.f;
    const uint32_t w = pack_bf16(x, y);
    pk[c / 2] = w;
    s0 += __uint_as_float(w << 16);
    s1 += __uint_as_float(w & 0xffff0000u);
  }
  tmem_st32(paddr, pk);
  return (s0 + s1) * kUnlift;
}

// the two warps of a lane quarter share its rows: barriers 1-4, 64 threads
__device__ __forceinline__ void pair_sync(int quarter) {
  __syncwarp();
  asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(quarter + 1) : "memory");
}
// whether `x` holds in any thread of the pair, once both warps have come here (and read S)
__device__ __forceinline__ bool any_row(bool x, int quarter) {
  uint32_t r;
  tc_fence_before();
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(x ? 1u : 0u), "r"(quarter + 1) : "memory");
  tc_fence_after();
  return r != 0;
}

// ------------------------------------------------------------------ kernel
// grid (S, row tiles, B*Hkv), cluster (S, 1, 1)
template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
k_attn_quant_tc(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const __grid_constant__ CUtensorMap tmap_kc, const __grid_constant__ CUtensorMap tmap_vc,
                AttnQuantParams p) {
  constexpr int UO = DH / 64;              // ring slots of K, and of V, of an own-block tile
  constexpr int LR = DH / 8;               // lanes of a row of Q
  constexpr int OC = DH / 2;               // output columns of a row's thread
  constexpr int kRowB = 2 * DH + 16;       // one share's partial row as sent to its owner
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  Bars& bars = *reinterpret_cast<Bars*>(smem + OFF_BAR);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int S = static_cast<int>(gridDim.x);
  const int r0 = blockIdx.y * BM;
  const int kvh = blockIdx.z % p.Hkv;
  const int G = p.Hq / p.Hkv;
  const int NT = p.NB * p.Dmax;
  int b = blockIdx.z / p.Hkv;

  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    prefetch_tmap(&tmap_kc);
    prefetch_tmap(&tmap_vc);
  }
  if (tid == 32) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&bars.full_k[s], 2);                      // the copy, and the tile's factors
      mbar_init(&bars.full_v[s], 1);
      mbar_init(&bars.empty_k[s], 1);
      mbar_init(&bars.empty_v[s], 1);
    }
    mbar_init(&bars.q_full, kSoftmax);
    mbar_init(&bars.recv_full, 1);
    mbar_init(&bars.v_clean, 1);
    mbar_init(&bars.o_done, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars.drained[i], 1);
    for (int i = 0; i < SLOTS; ++i) mbar_init(&bars.own_clean[i], kSoftmax);
    for (int i = 0; i < SBUF; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_free[i], 1);
      mbar_init(&bars.p_full[i], kSoftmax);
    }
    bars.failed = 0;
    bars.odd_own = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (p.longest_first) {
    // the CTAs of the longest prefixes start first
    int* lens = reinterpret_cast<int*>(smem);
    const int mine = tid < p.B ? p.prefix_len[tid] : -1;
    lens[tid] = mine;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < p.B; ++i) before += lens[i] > mine || (lens[i] == mine && i < tid) ? 1 : 0;
    if (tid < p.B && before == b) bars.seq = tid;
    __syncthreads();
    b = bars.seq;
  }
  // ends of the blocks in the list of present tokens, by one warp
  int* ends = reinterpret_cast<int*>(smem + OFF_K);
  if (warp == 0) {
    int sum = 0;
    for (int k0 = 0; k0 < p.NB; k0 += 32) {
      const int k = k0 + lane;
      int n = k < p.NB ? min(max(p.blk_len[static_cast<int64_t>(b) * p.NB + k], 0), p.Dmax) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += up;
      }
      if (k < p.NB) ends[k] = sum + n;
      sum += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) bars.rows = sum * G;
    fence_async_smem();                    // tensor copies write the same place later
  }
  int P = p.prefix_len[b];
  if (P < 0 || P > p.capacity) {
    if (tid == 0) record_error(p.hdr, SSD_ERR_DEVICE, 450);
    P = 0;
  }
  __syncthreads();
  const int rows_total = bars.rows;
  if (r0 >= rows_total) return;            // every CTA of the cluster
  const int rv = min(BM, rows_total - r0);
  if (tid < BM) {
    // slot of this row's token: the block whose end is the first above its number
    const int i = (r0 + min(tid, rv - 1)) / G;
    int lo = 0, hi = p.NB - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > i) hi = mid; else lo = mid + 1;
    }
    const int found = lo * p.Dmax + i - (lo > 0 ? ends[lo - 1] : 0);
    const int slot = in_range(found, NT, p.hdr, 454) ? found : 0;
    bars.row_slot[tid] = slot;
    bars.row_at[tid] = slot * p.Hq + kvh * G + (r0 + min(tid, rv - 1)) % G;
  }
  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();                         // the block ends have been read: the ring may be filled
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;

  // candidate slots of this row tile: from its first token's block on
  const int s_base = bars.row_slot[0] / p.Dmax * p.Dmax;
  const int s_end = bars.row_slot[rv - 1] + 1;
  const int own_tiles = (s_end - s_base + BN - 1) / BN;
  const int nC = rank == 0 ? own_tiles : 0;
  // prefix tiles of this rank; rank 0 takes two fewer for each own-block tile (masked: about
  // twice the work of a prefix tile)
  const int T = (P + BN - 1) / BN;
  int j0 = 0, j1 = T;
  if (S > 1) {
    const int first = min(T, max(0, (T + 2 * own_tiles + S - 1) / S - 2 * own_tiles)), rest = T - first;
    j0 = rank == 0 ? 0 : first + rest * (rank - 1) / (S - 1);
    j1 = rank == 0 ? first : first + rest * rank / (S - 1);
  }
  const int nP = j1 - j0, nT = nC + nP;
  const bool ragged = nP > 0 && j1 * BN > P;             // the last tile ends past the prefix
  // rows merged by this CTA: [rb, rb + nr)
  const int rpc = (rv + S - 1) / S;
  const int rb = rank * rpc, nr = max(0, min(rv, rb + rpc) - rb);
  float m = -INFINITY, l = 0.f;            // reference maximum (log2 units) and sum of a softmax row

  const bool softmax = warp < 4 || warp >= 8;
  const int half = warp < 4 ? 0 : 1;                       // columns 64 half .. of every tile
  const int row = (warp & 3) * 32 + lane;                  // TMEM lane
  if (softmax) {
    // ---------------------------------------------------------- rows
    const bool row_ok = row < rv;
    const int slot = bars.row_slot[row];
    const int c_lo = slot / p.Dmax * p.Dmax;
    // Q: a power of two brings a row's largest magnitude into [128, 256); two e4m3 parts. DH / 8
    // lanes take a row, a warp 16 rows four passes a round (a loop: this code runs once a CTA,
    // and unrolled it cost more in instruction fetches than in work).
    constexpr int kStep = 32 / LR, kPasses = 16 / kStep;
    const int q_row = ((warp & 3) + 4 * half) * 16 + lane / LR, chunk = lane % LR;
    const uint16_t* q_seq = p.q + static_cast<int64_t>(b) * NT * p.Hq * DH + chunk * 8;
    uint4 raw[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = q_row + kStep * i;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rv) raw[i] = *reinterpret_cast<const uint4*>(q_seq + static_cast<int64_t>(bars.row_at[r]) * DH);
    }
#pragma unroll 1
    for (int first = q_row; first < q_row + 16; first += 4 * kStep) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = first + kStep * i;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
#pragma unroll
        for (int o = 1; o < LR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = static_cast<int>(top >> 23);
        const int up = min(254 + 7 - ex, 253);
        const float mul = ex == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(up) << 23);
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(w[e] << 16) * mul;            // a row that is not finite becomes NaN
          x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * mul;
        }
        const uint32_t lo = e4m3x4(x[0], x[1], x[2], x[3]), hi = e4m3x4(x[4], x[5], x[6], x[7]);
        e4m3x2_to_f32(lo, y[0], y[1]);
        e4m3x2_to_f32(lo >> 16, y[2], y[3]);
        e4m3x2_to_f32(hi, y[4], y[5]);
        e4m3x2_to_f32(hi >> 16, y[6], y[7]);
        uint8_t* at = smem + OFF_Q8 + r * 128 + (((chunk >> 1) ^ (r & 7)) << 4) + (chunk & 1) * 8;
        *reinterpret_cast<uint2*>(at) = make_uint2(lo, hi);
        *reinterpret_cast<uint2*>(at + kSlot) = make_uint2(e4m3x4(x[0] - y[0], x[1] - y[1], x[2] - y[2], x[3] - y[3]),
                                                           e4m3x4(x[4] - y[4], x[5] - y[5], x[6] - y[6], x[7] - y[7]));
        if (nC > 0)
          *reinterpret_cast<uint4*>(smem + OFF_QB + (chunk >> 3) * kSlot + r * 128 + (((chunk & 7) ^ (r & 7)) << 4)) = raw[i];
        if (chunk == 0)
          bars.pair[0][r] = ex == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(254 - up) << 23) * p.scale_log2;
      }
#pragma unroll
      for (int i = 0; i + 4 < kPasses; ++i) raw[i] = raw[4 + i];
    }
    fence_async_smem();
    mbar_arrive(&bars.q_full);
    mbar_wait(bars, &bars.q_full, 0, p.hdr, 464);            // the factors of all rows are there
    const float q_mul = bars.pair[0][row];
    pair_sync(warp & 3);                                     // the pairs may be written again
    // Where a reference has to move: the row's new one, from both halves, and O and the sum
    // under it (each half rescales its columns of O).
    auto move_refs = [&](int j, float mx) {
      bars.pair[half][row] = mx;
      pair_sync(warp & 3);
      const float m_new = fmaxf(m, fmaxf(mx, bars.pair[half ^ 1][row]));
      const bool need = m_new > m + kLag;
      const float alpha = need ? ex2_approx(m - m_new) : 1.f;
      if (need) m = m_new;
      l *= alpha;
      pair_sync(warp & 3);                                    // the pairs may be written again
      if (j > 0 && __any_sync(0xffffffffu, need)) {
        // O holds the sum up to tile j - 1: wait for its last product, then rescale
        mbar_wait(bars, &bars.s_free[(j - 1) % SBUF], ((j - 1) / SBUF) & 1, p.hdr, 461);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int q = UO * half; q < UO * half + UO; ++q) {
          uint32_t o[32];
          tmem_ld32(tmem + TM_O + lane_off + q * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(tmem + TM_O + lane_off + q * 32, o);
        }
      }
    };
    uint32_t v[64];
    // ---- own-block tiles
    bool odd = false;
    for (int j = 0; j < nC; ++j) {
      // slots of other blocks and of absent tokens may hold anything, and 0 * inf is not 0:
      // values that are not finite leave the tile, and the rows that see one get it at the end. Eight
      // lanes read a value row; their largest magnitude is its scale.
      constexpr int kReads = BN * 8 / kSoftmax;
      uint32_t tops[kReads] = {};
      for (int h = 0; h < UO; ++h) {
        const int u = UO * j + h;
        if (!__all_sync(0xffffffffu, mbar_wait(bars, &bars.full_v[u % SLOTS], (u / SLOTS) & 1, p.hdr, 473))) break;
        uint4* vt = reinterpret_cast<uint4*>(smem + OFF_V + (u % SLOTS) * kSlot);
#pragma unroll
        for (int n = 0; n < kReads; ++n) {
          const int i = half * BM + row + n * kSoftmax;
          uint4 x = vt[i];
          uint32_t* w = reinterpret_cast<uint32_t*>(&x);
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((w[e] & 0x7f80u) == 0x7f80u) {
              w[e] &= 0xffff0000u;
              bad = true;
            }
            if ((w[e] & 0x7f800000u) == 0x7f800000u) {
              w[e] &= 0xffffu;
              bad = true;
            }
          }
          if (bad) {
            vt[i] = x;
            odd = true;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) tops[n] = max_u16x2(tops[n], w[e] & 0x7fff7fffu);
        }
      }
#pragma unroll
      for (int n = 0; n < kReads; ++n) {
        uint32_t top = max(tops[n] & 0xffffu, tops[n] >> 16);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((lane & 7) == 0) bars.own_lv[j & 1][(half * BM + row + n * kSoftmax) >> 3] = own_scale_log2(top);
      }
      if (odd) *reinterpret_cast<volatile int*>(&bars.odd_own) = 1;
      fence_async_smem();
      mbar_arrive(&bars.own_clean[j % SLOTS]);
      const int sb = j % SBUF;
      mbar_wait(bars, &bars.s_full[sb], (j / SBUF) & 1, p.hdr, 460);
      __syncwarp();
      tc_fence_after();
      const uint32_t sp = tmem + TM_S + sb * BN + lane_off;
      load64(sp + half * 64, v);
      const int s0 = s_base + j * BN + half * 64;
      const int lo = row_ok ? c_lo - s0 : BN, hi = row_ok ? slot + 1 - s0 : 0;
      // every softmax thread's scales are there (they are written again two tiles on, behind the next
      // tile's barrier)
      __syncwarp();
      asm volatile("barrier.cta.sync.aligned 5, %0;" ::"n"(kSoftmax) : "memory");
      const float mx = own_max(v, p.scale_log2, bars.own_lv[j & 1] + half * 64, lo, hi);
      if (any_row(mx > m + kLag, warp & 3)) move_refs(j, mx);
      l += chunk_pairs(v, sp + half * 32, p.scale_log2, lo, hi, m == -INFINITY ? 0.f : m);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars.p_full[sb]);
    }
    // ---- prefix tiles
    for (int t = j0; t < j1; ++t) {
      const int j = nC + t - j0, sb = j % SBUF;
      mbar_wait(bars, &bars.s_full[sb], (j / SBUF) & 1, p.hdr, 460);
      __syncwarp();
      tc_fence_after();
      const uint32_t sp = tmem + TM_S + sb * BN + lane_off;
      // the factors were written before the tile's products were issued
      const float4(&ft)[3][2] = bars.factors[(t - j0) % FACTORS];
      const float4 fk = ft[0][half], fl = ft[1][half], fw = ft[2][half];
      const Groups f = {{fk.x * q_mul, fk.y * q_mul, fk.z * q_mul, fk.w * q_mul}, {fl.x, fl.y, fl.z, fl.w}, {fw.x, fw.y, fw.z, fw.w}};
      load64(sp + half * 64, v);
      const int hi = P - t * BN - half * 64;
      const bool full = P - t * BN >= BN;
      const float mx = full ? chunk_max<false>(v, f, 0) : chunk_max<true>(v, f, hi);
      if (any_row(mx > m + kLag, warp & 3)) move_refs(j, mx);
      const float ref = m == -INFINITY ? 0.f : m;
      l += full ? chunk_parts<false>(v, sp + half * 16, f, 0, ref) : chunk_parts<true>(v, sp + half * 16, f, hi, ref);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars.p_full[sb]);
    }
    bars.pair[half][row] = l;                              // read after the barrier before the merge
    if (nT > 0) mbar_wait(bars, &bars.o_done, 0, p.hdr, 462);
    __syncwarp();
    tc_fence_after();
  } else if (warp == 4 || warp == 6) {
    // ---------------------------------------------------------- producers (4: K, 6: V)
    // Unit u goes to slot u % SLOTS: the two halves of an own-block tile, or a prefix tile. Lanes
    // 0-15 of the K side also fetch a prefix tile's K and V scales, two tiles ahead of the copy
    // (and the page a tile ahead of them), and leave the factors made of them in shared memory:
    // a tile's products, whose end the softmax waits for, start only after them. Their place is
    // free by then: this copy's slot was left by the products of the tile four before, which
    // waited for the softmax of the tile seven before.
    const bool kside = warp == 4;
    uint64_t* full = kside ? bars.full_k : bars.full_v;
    uint64_t* empty = kside ? bars.empty_k : bars.empty_v;
    const uint32_t ring = sbase + (kside ? OFF_K : OFF_V);
    // whether the slot of unit u may be filled: no more copies once a wait gave up
    auto slot_for = [&](int u) -> bool {
      if (u >= SLOTS) mbar_wait(bars, &empty[u % SLOTS], ((u / SLOTS) - 1) & 1, p.hdr, kside ? 470 : 471);
      return __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&bars.failed), 0) == 0;
    };
    int u = 0;
    bool go = true;
    for (int j = 0; go && j < nC; ++j) {
      for (int h = 0; h < UO; ++h, ++u) {
        if (!(go = slot_for(u))) break;
        if (lane == 0) {
          if (kside) mbar_arrive(&full[u % SLOTS]);        // no factors
          mbar_expect_tx(&full[u % SLOTS], kSlot);
          tma_load_3d(ring + (u % SLOTS) * kSlot, kside ? &tmap_kc : &tmap_vc, 64 * h, kvh, b * NT + s_base + j * BN,
                      &full[u % SLOTS]);
        }
      }
    }
    auto load_page = [&](int t) -> int {
      if (t >= j1 || p.block_table == nullptr) return b;
      if (!in_range(t, p.pages_per_seq, p.hdr, 452)) return 0;
      const int pg = p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + t];
      if (pg >= 0 && pg < p.num_pages) return pg;
      if (lane == 0) record_error(p.hdr, SSD_ERR_DEVICE, 451);
      return 0;
    };
    const int blocks = static_cast<int>(p.blocks);
    auto load_scale = [&](int t, int pg) -> float {
      if (!kside || t >= j1 || lane >= 16) return 0.f;
      const int place = (p.block_table == nullptr ? t * BN : 0) + (lane & 7) * 16;
      const int blk = min(place >> p.sb_log2, blocks - 1);
      if (!in_range(static_cast<int64_t>(pg * p.Hkv + kvh) * blocks + blk, p.num_pages * p.Hkv * blocks, p.hdr, 453)) return 0.f;
      return (lane < 8 ? p.k_scale : p.v_scale)[static_cast<int64_t>(pg * p.Hkv + kvh) * blocks + blk];
    };
    int page = load_page(j0), page1 = load_page(j0 + 1), page2 = load_page(j0 + 2);
    float scale = load_scale(j0, page), scale1 = load_scale(j0 + 1, page1);
    for (int t = j0; go && t < j1; ++t, ++u) {
      if (!(go = slot_for(u))) break;
      if (lane == 0) {
        mbar_expect_tx(&full[u % SLOTS], kSlot);
        tma_load_2d(ring + (u % SLOTS) * kSlot, kside ? &tmap_k : &tmap_v, 0,
                    (page * p.Hkv + kvh) * static_cast<int>(p.page_tokens) + (p.block_table == nullptr ? t * BN : 0),
                    &full[u % SLOTS]);
      }
      if (kside) {
        float* at = reinterpret_cast<float*>(bars.factors[(t - j0) % FACTORS]);
        if (lane < 8) {
          at[lane] = scale;
        } else if (lane < 16) {
          const float lv = fmaxf(__log2f(scale), kLeastVScaleLog2);
          at[lane] = lv;
          at[lane + 8] = ex2_approx(-lv);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[u % SLOTS]);
      }
      scale = scale1;
      scale1 = load_scale(t + 2, page2);
      page = page1;
      page1 = page2;
      page2 = load_page(t + 3);
    }
    if (lane == 0) bars.sent[kside ? 0 : 1] = u;
    __syncwarp();
    if (!kside && ragged) {
      const int u = UO * nC + nP - 1;
      if (mbar_wait(bars, &full[u % SLOTS], (u / SLOTS) & 1, p.hdr, 472)) {
        uint4* v = reinterpret_cast<uint4*>(smem + OFF_V + (u % SLOTS) * kSlot);
        for (int i = (P - (j1 - 1) * BN) * 8 + lane; i < BN * 8; i += 32) v[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.v_clean);
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------- S = Q K^T
    // Descriptors of one operand differ in the address field alone (16-byte units, no carry out
    // of it): one base and small sums keep the issue ahead of the tensor pipe's 64 clocks a product.
    if (lane == 0 && nT > 0) {
      constexpr uint32_t idS = idesc_f8(false, false, BN), idSb = idesc_bf16(false, BN);
      const uint64_t q8 = sw128_desc(sbase + OFF_Q8, 16, 1024), qb = sw128_desc(sbase + OFF_QB, 16, 1024),
                     k0 = sw128_desc(sbase + OFF_K, 16, 1024);
      mbar_wait(bars, &bars.q_full, 0, p.hdr, 480);
      int u = 0;
      for (int j = 0; j < nT; ++j) {
        const int sb = j % SBUF;
        const uint32_t d = tmem + TM_S + sb * BN;
        const bool own = j < nC;
        const int s0 = u % SLOTS, s1 = (u + UO - 1) % SLOTS;
        // the buffer still holds P of tile j - SBUF until its product is done
        if (j >= SBUF) mbar_wait(bars, &bars.s_free[sb], (j / SBUF - 1) & 1, p.hdr, 483);
        mbar_wait(bars, &bars.full_k[s0], (u / SLOTS) & 1, p.hdr, 481);
        if (own) mbar_wait(bars, &bars.full_k[s1], ((u + UO - 1) / SLOTS) & 1, p.hdr, 482);
        tc_fence_after();
        const uint64_t kd = k0 + static_cast<uint32_t>(s0) * (kSlot / 16);
        if (own) {
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks)
            mma_bf16(d, qb + (ks >> 2) * (kSlot / 16) + (ks & 3) * 2, kd + (ks >> 2) * (kSlot / 16) + (ks & 3) * 2, idSb,
                     ks > 0 ? 1u : 0u);
        } else {
#pragma unroll
          for (int ks = 0; ks < DH / 32; ++ks) {
            mma_f8(d, q8 + ks * 2, kd + ks * 2, idS, ks > 0 ? 1u : 0u);
            mma_f8(d, q8 + kSlot / 16 + ks * 2, kd + ks * 2, idS, 1u);
          }
        }
        mma_commit(&bars.s_full[sb]);
        mma_commit(&bars.empty_k[s0]);
        if (own && UO > 1) mma_commit(&bars.empty_k[s1]);
        u += own ? UO : 1;
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- O += P V (warp 7)
    if (lane == 0 && nT > 0) {
      // rows of codes are 128 bytes in the ring, zeros behind a shorter head's
      constexpr uint32_t idPV = idesc_f8(true, true, 128), idPVb = idesc_bf16(true, DH);
      const uint64_t v0 = sw128_desc(sbase + OFF_V, kSlot, 1024);
      int u = 0;
      for (int j = 0; j < nT; ++j) {
        const int sb = j % SBUF;
        const bool own = j < nC;
        const int s0 = u % SLOTS, s1 = (u + UO - 1) % SLOTS;
        mbar_wait(bars, &bars.full_v[s0], (u / SLOTS) & 1, p.hdr, 484);
        if (own) {
          mbar_wait(bars, &bars.full_v[s1], ((u + UO - 1) / SLOTS) & 1, p.hdr, 485);
          mbar_wait(bars, &bars.own_clean[j % SLOTS], (j / SLOTS) & 1, p.hdr, 487);
        }
        if (ragged && j == nT - 1) mbar_wait(bars, &bars.v_clean, 0, p.hdr, 486);
        mbar_wait(bars, &bars.p_full[sb], (j / SBUF) & 1, p.hdr, 488);
        tc_fence_after();
        const uint64_t vd = v0 + static_cast<uint32_t>(s0) * (kSlot / 16);
        const uint32_t pa = tmem + TM_S + sb * BN;
        if (own) {
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            mma_bf16_ts(tmem + TM_O, pa + ks * 8, vd + ks * (16 * 128 / 16), idPVb, (j > 0 || ks > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int ks = 0; ks < BN / 32; ++ks) {
            mma_f8_ts(tmem + TM_O, pa + ks * 8, vd + ks * (32 * 128 / 16), idPV, (j > 0 || ks > 0) ? 1u : 0u);
            mma_f8_ts(tmem + TM_O, pa + PART + ks * 8, vd + ks * (32 * 128 / 16), idPV, 1u);
            mma_f8_ts(tmem + TM_O, pa + 2 * PART + ks * 8, vd + ks * (32 * 128 / 16), idPV, 1u);
          }
        }
        mma_commit(&bars.s_free[sb]);
        mma_commit(&bars.empty_v[s0]);
        if (own && UO > 1) mma_commit(&bars.empty_v[s1]);
        u += own ? UO : 1;
        // the two kinds of products into O: the order between them is made
        if (own) {
          mbar_wait(bars, &bars.s_free[sb], (j / SBUF) & 1, p.hdr, 489);
          tc_fence_after();
        }
      }
      mma_commit(&bars.o_done);
    }
    __syncwarp();
  }

  // After a wait gave up (every role has ended): this CTA's copies and products still in flight are
  // given as long again before shared memory serves another purpose, TMEM is freed and the CTA ends.
  auto drain = [&] {
    if (lane != 0 || !bars.failed) return;
    int gave_up = 0;
    if (warp == 4 || warp == 6) {
      const int n = bars.sent[warp == 4 ? 0 : 1];
      for (int i = max(0, n - SLOTS); i < n; ++i)
        mbar_wait_bounded((warp == 4 ? bars.full_k : bars.full_v) + i % SLOTS, (i / SLOTS) & 1, &gave_up, p.hdr, 491, kWaitClocks);
    } else if (warp == 5 || warp == 7) {
      uint64_t* bar = &bars.drained[warp == 5 ? 0 : 1];
      mma_commit(bar);
      mbar_wait_bounded(bar, 0, &gave_up, p.hdr, 492, kWaitClocks);
    }
  };

  // ---- one share: the rows leave from TMEM
  if (S == 1) {
    if (softmax) {
      pair_sync(warp & 3);                                   // both halves' sums are there
      const int slot = bars.row_slot[row];
      const float inv = __frcp_rn(bars.pair[0][row] + bars.pair[1][row]);
      const bool look = nC > 0 && *reinterpret_cast<volatile int*>(&bars.odd_own);
      const int64_t at = (static_cast<int64_t>(b) * NT * p.Hq + bars.row_at[row]) * DH + half * OC;
#pragma unroll 1
      for (int q = 0; q < UO; ++q) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(tmem + TM_O + lane_off + half * OC + q * 32, o);
        tmem_wait_ld();
        if (row >= rv || bars.failed) continue;
        if (!in_range(at + q * 32 + 31, static_cast<int64_t>(p.B) * NT * p.Hq * DH, p.hdr, 455)) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * kUnlift * inv);
        if (look) {
          // the own-block values that left the tile: an infinity or NaN, whatever its weight
          for (int t = slot / p.Dmax * p.Dmax; t <= slot; ++t) {
            const uint16_t* v = p.v_cand + ((static_cast<int64_t>(b) * NT + t) * p.Hkv + kvh) * DH + half * OC + q * 32;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((v[e] & 0x7f80u) == 0x7f80u) o[e] = __float_as_uint(__uint_as_float(o[e]) + bf16_to_f32(v[e]));
          }
        }
        if (p.out_f32) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at + q * 32);
#pragma unroll
          for (int u = 0; u < 8; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at + q * 32);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16(__uint_as_float(o[8 * u + 2 * e]), __uint_as_float(o[8 * u + 2 * e + 1]));
            dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
    }
    __syncthreads();
    if (bars.failed) {
      drain();
      __syncthreads();
    }
    if (warp == 4) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
    return;
  }

  // ---- merge the S shares of every row in the CTA that owns it. Ring layout (bytes): staged
  // rows [BM][kRowB], received rows [sender][rpc][kRowB].
  uint8_t* stage = smem + OFF_K;
  uint8_t* recv = stage + BM * kRowB;
  auto part = [&](int c, int i) -> const uint8_t* {
    return c == rank ? stage + (rb + i) * kRowB : recv + (c * rpc + i) * kRowB;
  };
  if (softmax) {
    const uint32_t oa = tmem + TM_O + lane_off + half * OC;
    pair_sync(warp & 3);                                        // both halves' sums are there
    uint32_t o[OC];
    if (nT > 0) {
#pragma unroll
      for (int c = 0; c < OC; c += 32) tmem_ld32(oa + c, o + c);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int e = 0; e < OC; ++e) o[e] = 0u;
    }
    float amax = 0.f;
    bool odd = false;                                    // an element is not finite
#pragma unroll
    for (int e = 0; e < OC; ++e) {
      odd |= (o[e] & 0x7f800000u) == 0x7f800000u;
      amax = fmaxf(amax, fabsf(__uint_as_float(o[e])));
    }
    if (odd) {
      amax = 0.f;
#pragma unroll
      for (int e = 0; e < OC; ++e)
        if ((o[e] & 0x7f800000u) != 0x7f800000u) amax = fmaxf(amax, fabsf(__uint_as_float(o[e])));
    }
    const int k = (amax >= 0x1p-100f) ? static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127 : -1;
    const int ex = min(k, 125) + 1;
    const float scale = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);
    const float inv_scale = __uint_as_float(static_cast<uint32_t>(127 - 14 - static_cast<int>(kLift) + ex) << 23);
    uint4* dst = reinterpret_cast<uint4*>(stage + row * kRowB + half * DH);
#pragma unroll
    for (int u = 0; u < OC / 8; ++u) {
      uint32_t pk[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = o[8 * u + 2 * e], y = o[8 * u + 2 * e + 1];
        pk[e] = pack_i16(__uint_as_float(x), __uint_as_float(y), scale);
        if (odd) {                                       // -2^15 stands for what is not finite
          if ((x & 0x7f800000u) == 0x7f800000u) pk[e] = (pk[e] & 0xffff0000u) | 0x8000u;
          if ((y & 0x7f800000u) == 0x7f800000u) pk[e] = (pk[e] & 0xffffu) | 0x80000000u;
        }
      }
      dst[u] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
    float* tail = reinterpret_cast<float*>(stage + row * kRowB + 2 * DH);
    if (half == 0) {
      tail[0] = m;
      // a share that gave up makes the rows NaN
      tail[1] = *reinterpret_cast<volatile int*>(&bars.failed) ? NAN : l + bars.pair[1][row];
    }
    // the sign tells the owner of the row to look closer
    const bool look = odd || (nC > 0 && *reinterpret_cast<volatile int*>(&bars.odd_own));
    tail[2 + half] = look ? -inv_scale : inv_scale;
    fence_async_smem();
  }
  if (tid == 0) mbar_expect_tx(&bars.recv_full, static_cast<uint32_t>((S - 1) * nr * kRowB));
  tc_fence_before();
  __syncwarp();
  cluster_sync();                                        // every ring of the cluster is idle
  tc_fence_after();
  if (bars.failed) drain();
  if (tid < S - 1) {
    const int c = (rank + 1 + tid) % S;
    const int n_c = min(rv, (c + 1) * rpc) - c * rpc;
    if (n_c > 0) {
      const uint32_t dst = map_peer(smem_u32(recv + rank * rpc * kRowB), static_cast<uint32_t>(c));
      const uint32_t bar = map_peer(smem_u32(&bars.recv_full), static_cast<uint32_t>(c));
      bulk_copy_to_peer(dst, smem_u32(stage + c * rpc * kRowB), static_cast<uint32_t>(n_c * kRowB), bar);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  __syncthreads();
  for (int it = tid; it < nr * (DH / 16); it += kThreads) {
    const int i = it / (DH / 16), cg = it % (DH / 16);
    if (!mbar_wait(bars, &bars.recv_full, 0, p.hdr, 490)) continue;
    // the shares under their common maximum; one without keys has sum 0 and zeros, and a NaN score
    // leaves the maximum and is in the sum
    float M = -INFINITY, L = 0.f;
    for (int c = 0; c < S; ++c) M = fmaxf(M, *reinterpret_cast<const float*>(part(c, i) + 2 * DH));
    bool look = false;
    float acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int c = 0; c < S; ++c) {
      const uint8_t* pr = part(c, i);
      const float4 tl = *reinterpret_cast<const float4*>(pr + 2 * DH);
      const uint4* src = reinterpret_cast<const uint4*>(pr + cg * 32);
      const uint4 h0 = src[0], h1 = src[1];
      const float f = tl.x > -INFINITY ? ex2_approx(tl.x - M) : 1.f, unit = cg < DH / 32 ? tl.z : tl.w;
      L = fmaf(tl.y, f, L);
      look |= unit < 0.f;
      const float g = f * fabsf(unit);
      const uint32_t w[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 v = unpack_i16(w[e]);
        acc[2 * e] = fmaf(g, v.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(g, v.y, acc[2 * e + 1]);
      }
    }
    if (bars.failed) continue;
    const float inv = __frcp_rn(L);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] *= inv;
    const int slot = bars.row_slot[rb + i];
    if (look) {
      for (int c = 0; c < S; ++c) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(part(c, i) + cg * 32);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if ((w[e] & 0xffffu) == 0x8000u) acc[2 * e] = NAN;
          if ((w[e] >> 16) == 0x8000u) acc[2 * e + 1] = NAN;
        }
      }
      // the own-block values that left the tile: an infinity or NaN, whatever its weight
      for (int t = slot / p.Dmax * p.Dmax; t <= slot; ++t) {
        const uint16_t* v = p.v_cand + ((static_cast<int64_t>(b) * NT + t) * p.Hkv + kvh) * DH + cg * 16;
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if ((v[e] & 0x7f80u) == 0x7f80u) acc[e] += bf16_to_f32(v[e]);
      }
    }
    const int64_t at = (static_cast<int64_t>(b) * NT * p.Hq + bars.row_at[rb + i]) * DH + cg * 16;
    if (!in_range(at + 15, static_cast<int64_t>(p.B) * NT * p.Hq * DH, p.hdr, 456)) continue;
    if (p.out_f32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
      for (int u = 0; u < 4; ++u) o[u] = make_float4(acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]);
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
      o[0] = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                        pack_bf16(acc[6], acc[7]));
      o[1] = make_uint4(pack_bf16(acc[8], acc[9]), pack_bf16(acc[10], acc[11]), pack_bf16(acc[12], acc[13]),
                        pack_bf16(acc[14], acc[15]));
    }
  }
  // this CTA's outgoing copies have finished reading its staged rows before it exits
  if (tid < S - 1) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  if (tid == 0 && nr > 0 && bars.failed) {               // ... and the incoming ones have arrived
    int gave_up = 0;
    mbar_wait_bounded(&bars.recv_full, 0, &gave_up, p.hdr, 493, kWaitClocks);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------------ host
static bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
                     const cuuint64_t* strides, const cuuint32_t* box) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Kernel attributes, once a device, and how many clusters of S CTAs are resident at once.
template <int DH>
static int resident(int S) {
  static std::mutex mu;
  static bool ready[kMaxDevices];
  static int found[kMaxDevices][kMaxSplit + 1];
  const int dev = current_device();
  if (dev < 0) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(k_attn_quant_tc<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes)) !=
            cudaSuccess ||
        cudaFuncSetAttribute(k_attn_quant_tc<DH>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    for (int n = 1; n <= kMaxSplit; ++n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(n), 1, 1);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kSmemBytes;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(n);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int count = 0;
      if (cudaOccupancyMaxActiveClusters(&count, k_attn_quant_tc<DH>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        count = 0;
      }
      found[dev][n] = count;
    }
    ready[dev] = true;
  }
  return found[dev][S];
}

// CTAs that share a row tile's prefix: those whose waves of resident clusters cost least. A CTA takes its
// share of the longest prefix's tiles and the time of 14 for its start and merge. The host knows
// only the capacity: where prefixes are equal waves count in full, where they vary (the longest
// started first) by the work, so the mean of both is taken. us by 1 .. 6 CTAs, 8 kv heads, replayed
// from a graph, cold: 320 rows of one sequence of 4096 keys 54.4 38.0 31.9 29.8 *27.8 42.1, of 4 *56.4 68.7
// 81.0 74.9 87.2 97.4; 120 rows of 16 sequences of 1k-16k 146.6 *115.8 126.1 138.4 154.8 169.1, of
// 4096 *57.5 75.0 89.2 101.5 111.7 124.0 (* the one taken); 800 rows of 4 of 32768 571 *468 532, of 2 of
// 8192 93 *106 118 (one wave would do, but equal lengths are not known here). Few row tiles over a
// long prefix take up to 16 (one of 32768, 2 kv heads, 320 rows: 40 us; with 8, 54).
template <int DH>
static int choose_split(long long groups, long long tiles) {
  int best = 0;
  double cost = 0;
  for (int S = 1; S <= kMaxSplit && S <= std::max<long long>(tiles, 1); ++S) {
    const int clusters = resident<DH>(S);
    if (clusters <= 0) continue;
    const double waves = static_cast<double>(groups) / clusters;
    const double c = (static_cast<double>(tiles) / S + 14.) * (std::ceil(waves) + std::max(1., 0.8 * waves)) / 2;
    if (best == 0 || c < 0.95 * cost) {
      cost = c;
      best = S;
    }
  }
  return best;
}

}  // namespace qtc

bool attn_quant_tc_applies(const AttnQuantParams& p) {
  if (p.NB > qtc::kMaxBlocks) return false;
  if (static_cast<long long>(p.NB) * p.Dmax * p.Hq >= (1LL << 31)) return false;
  if (static_cast<long long>(p.B) * p.Hkv > 65535 || static_cast<long long>(p.B) * p.NB * p.Dmax >= (1LL << 31)) return false;
  return tc::encode_fn() != nullptr;
}

template <int DH>
static int tc_launch(const AttnQuantParams& p, cudaStream_t s) {
  using namespace qtc;
  const int NT = p.NB * p.Dmax;
  const int G = p.Hq / p.Hkv;
  const int mtiles = (NT * G + BM - 1) / BM;
  const int S = choose_split<DH>(static_cast<long long>(p.B) * p.Hkv * mtiles, (p.capacity + BN - 1) / BN + 2);
  if (S < 1) return SSD_ERR_CUDA;
  // an empty cache is never read, but a map needs an address and a row
  const uint64_t rows = static_cast<uint64_t>(p.num_pages) * p.Hkv * p.page_tokens;
  const void *kb = rows > 0 ? p.k_cache : static_cast<const void*>(p.q), *vb = rows > 0 ? p.v_cache : kb;
  const cuuint64_t dims2[2] = {DH, rows > 0 ? rows : 1}, strides2[1] = {DH};
  const cuuint32_t box2[2] = {128, BN};             // what lies past a shorter row is filled with zeros
  const cuuint64_t dims3[3] = {DH, static_cast<cuuint64_t>(p.Hkv), static_cast<cuuint64_t>(p.B) * NT};
  const cuuint64_t strides3[2] = {DH * 2, static_cast<cuuint64_t>(p.Hkv) * DH * 2};
  const cuuint32_t box3[3] = {64, 1, BN};
  CUtensorMap mk, mv, mkc, mvc;
  if (!make_map(&mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, kb, 2, dims2, strides2, box2) ||
      !make_map(&mv, CU_TENSOR_MAP_DATA_TYPE_UINT8, vb, 2, dims2, strides2, box2) ||
      !make_map(&mkc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.k_cand, 3, dims3, strides3, box3) ||
      !make_map(&mvc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.v_cand, 3, dims3, strides3, box3))
    return SSD_ERR_CUDA;
  AttnQuantParams q = p;
  q.longest_first = p.B > 1 && p.B <= kThreads ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(S), static_cast<unsigned>(mtiles), static_cast<unsigned>(p.B * p.Hkv));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
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
  if (cudaLaunchKernelEx(&cfg, k_attn_quant_tc<DH>, mk, mv, mkc, mvc, q) != cudaSuccess) {
    cudaGetLastError();
    return SSD_ERR_CUDA;
  }
  count_launch();
  return check_launch();
}

int attn_quant_tc_launch(const AttnQuantParams& p, int dh, cudaStream_t s) {
  return dh == 128 ? tc_launch<128>(p, s) : tc_launch<64>(p, s);
}

}  // namespace ssd
