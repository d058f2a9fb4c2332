// Sampling distributions of logit rows: temperature, top-k, top-p and min-p, as probability
// rows (ssd_filter_probs) and as tokens drawn by a given uniform number (ssd_sample).
//
// Weights w_i = 2^((z_i - z_max) log2(e) / T) are pairs of fp32 numbers (relative error under
// 2^-29) and, where they are summed, integers round(w_i 2^43): the sums are exact, so neither a
// cut nor a token depends on the order in which threads add. The tokens that stay are the first
// ones in the order (z descending, index ascending), so one composite number
//   comp = (okey(z_max) - okey(z)) * 2^20 + index       (okey: the fp32 order as unsigned integers)
// and one bound say which; ties at the border are thereby cut by their index.
//
// A cluster of 1 to 8 CTAs holds a row in its shared memory: it is read from HBM once, and every
// further pass reads shared memory. Partial results cross the cluster through distributed shared
// memory. Rows beyond the cluster's shared memory are read again from L2. The passes:
//   1  the largest value; with top-k also a value that at least k tokens reach (the share-th largest of
//      the warps' or the threads' own largest, the least of these over the CTAs);
//   2a top-k up to 1024: the tokens above that value, as a rule little more than k, are brought together
//      and sorted in every CTA; top-k, top-p, min-p and the draw follow from that list alone;
//   2b larger top-k: bins of the values from there up (count and weight), the tokens of the bin in
//      which the k-th lies sorted;
//   2c top-p alone, or behind 2b: all weights summed, those that can matter in 512 bins of their value;
//      the tokens of the bin in which the sum passes top_p of the whole sorted. Tokens of a weight
//      below (1 - top_p) / V cannot be the border and are not binned;
//   3  the weight of what stays, where min-p or a draw needs it; the output rows; the token.
// Lists too long to be sorted (thousands of equal values) go through `select`, nine bits of comp a level.
//
// What bounds it: not HBM. 81 rows of 128256 fp32 logits (nucleus) take 82-92 us, 0.9-1.0 TB/s of the 83 MB
// that have to be moved (12 us): about 90 instructions a token (two evaluations of its weight of 25
// each, the rest bins, tests and the output) and 2000 a warp for the fixed phases, barriers across a
// cluster of six among them; issue slots are busy for half of the time with two CTAs an SM, which is
// what registers (64 a thread) and shared memory allow. Clocks of a CTA's 88 thousand there: load 6, largest
// value 5, weights and bins 20, their sums and bin 9, the bin's tokens brought together and sorted 30 (other
// CTAs of the cluster waited for in that), cut 3, output 10. In steps (us, that case / 64 tokens of 151936
// bf16 logits): every level of a radix search weighs every token 221 / 245; one fp64 division and
// logarithm a thread taken out 219 / 163 (a single row 87 -> 17); bins of linear width 133 / 68; pairs
// of fp32 in one instruction 93; the border's tokens sorted in registers and the row on six CTAs
// instead of eight 85; top-k bounded from each warp's four largest (256 rows 66 -> 60) 82 / 69;
// top-k up to 1024 from the list 82 / 63; lists of more than 1024 tokens sorted a CTA each and merged 82 / 61.
// Tried without gain: 384 threads and no spilled registers; weights added to a bin by two additions
// that wait for nothing instead of one that returns its carry.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "ssd_kvq.cuh"
#include "ssd_tc.cuh"

namespace ssd {
namespace smp {

using tc::cluster_rank;
using tc::cluster_sync;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;                 // of one level of `select`
constexpr int kBinBits = 9;
constexpr int kLin = 512;                  // bins of a row's values, the first level of top-p
constexpr int kMaxCluster = 8;
constexpr int kIdxBits = 20;               // V <= 2^20: the weight sums then fit 64 bits
constexpr int kTab = 64;
constexpr uint64_t kAll = ~0ull;
constexpr int kTop = 4;                     // of each warp's lanes' largest, the ones that bound small top-k
// Up to kShortK the tokens above the bound are sorted, beyond they are binned. us by the list / by bins, top-k alone and with
// top-p 0.95: 64 rows of 151936 bf16 logits k 50 22 / 29, 22 / 59; 400 33 / 34, 34 / 64; 1000 46 / 41, 46 / 71; 1300 54 / 44,
// 84 / 73. 8 rows of 128256: 400 21 / 23, 22 / 39; 1000 26 / 24, 26 / 41. Where a CTA holds a whole row its list is too
// short from about 500 on, and what was brought together is binned after all: 300 rows of 32000 400 37 / 41, 37 / 66; 1000 62 / 51,
// 89 / 78.
constexpr int kShortK = 1024;
constexpr int kList = 1024;                // tokens near a border that one CTA may hold,
constexpr int kFew = kThreads;             // tokens from which one is drawn by sorting them once more
constexpr int kThreadTokens = 512;         // a thread's part of a row, at most
constexpr int kMerged = 4 * kThreads;      // and all CTAs of the cluster together, to be sorted

struct Params {
  const void* logits;
  int64_t row_bytes;
  int V;
  int64_t rows_per;                        // rows that share a setting
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const int32_t* blk_len;
  int NB, Dmax;
  const float* u;
  int32_t* token;
  float* prob;
  float* probs;
  int nvw, nres;                           // 16-byte vectors a warp owns, and those of them kept in shared memory
  WsHeader* hdr;
};

struct Shared {
  uint4 ends[2];
  float2 pow[kTab];                        // kPowers
  int2 tab[kTab];                          // powers of two of the row (make_table)
  union {
    uint32_t hist[2][4][kBins];            // count; sums of bits 0-15 (or 0-31), 16-31 and 32-43 of the weight; two levels in turns
    uint64_t sorted[kMerged];
  };
  uint64_t list[kList];                    // this CTA's tokens near a border
  uint64_t ex_sum[2][kMaxCluster];         // from every CTA of the cluster
  float ex_max[kMaxCluster];
  uint32_t ex_key[kMaxCluster];
  uint64_t part[kWarps], part2[kWarps];
  uint64_t wsum[kWarps];
  float wmax[kWarps];
  uint32_t wkey[kWarps * kTop];
  uint64_t sel_e, sel_incl;                // of the bin chosen: weight before it, and with it
  uint32_t sel_n, sel_cnt, sel_bin, list_n;
};

// the same variable in the CTA of rank `r`
template <typename T>
__device__ __forceinline__ T* peer(T* p, int r) {
  uint64_t out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(r));
  return reinterpret_cast<T*>(out);
}

__device__ __forceinline__ uint32_t okey(float z) {
  const uint32_t b = __float_as_uint(z);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float okey_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// 2^(i/64) as the nearest fp32 number h and what that lacks, 2^(i/64) / h - 1: the exponential's
// series in fp64, which ends below 2^-60 for x <= ln 2
struct Powers {
  float2 v[kTab];
  constexpr Powers() : v() {
    for (int i = 0; i < kTab; ++i) {
      const double x = 0.69314718055994530942 * i / kTab;
      double sum = 1., term = 1.;
      for (int k = 1; k < 20; ++k) {
        term = term * x / k;
        sum += term;
      }
      v[i].x = static_cast<float>(sum);
      v[i].y = static_cast<float>((sum - v[i].x) / v[i].x);
    }
  }
};
__device__ constexpr Powers kPowers;

constexpr float kFltMax = 3.402823466e38f;
constexpr float kMagic = 12582912.f;       // 1.5 * 2^23: adding it rounds to an integer, held in the low bits
constexpr int kMagicBits = 0x4B400000;

// two fp32 numbers in one register pair: one instruction for both, each rounded as alone
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
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Weights w = 2^((z - zmax) c), c = ch + cl = log2(e) / T, of z >= zmin (where w >= 2^-125.5).
// `plain` rows: with n = round(64 z ch), held in the low bits of m = 64 z ch + 1.5 2^23,
//   64 z c = n + r,  r = (64 z ch - n) + 64 z cl,   w = 2^(n/64 - zmax c) 2^(r/64)
// and the first factor is entry n mod 64 of a table of the row, 2^(i/64 - zmax c) with what its fp32
// number lacks, plus n / 64 in the exponent (the entry's bits are less i 2^17, so that the bits of m
// shifted by 17 are all there is to add). Values below zmin act as zmin, whose weight sums see as 0.
// Other rows: 64 |zmax c| >= 2^21 (m would lose bits), an infinity, or a zmin that is not far
// enough below zmax or not above -inf. They take differences to zmax first: where |zmax c| is
// large, every z >= zmin lies within a factor of two of it, so that these are exact again.
struct Scale {
  float zmax, zmin, c64, cl64, zp, mu;
  int nbias;
  uint32_t kmax;
  bool plain;
};

// what depends on the temperature alone, in pairs of fp32 numbers: a division in fp64 by every thread
// of a CTA takes microseconds here
struct Rate {
  float ch, cl, span;                      // log2(e) / T, and 125.49 of its inverse
};
__device__ __forceinline__ Rate make_rate(float temp) {
  Rate t;
  t.ch = fminf(__fdiv_rn(1.44269502f, temp), 0x1p120f);
  t.cl = t.ch < 0x1p120f ? __fdiv_rn(fmaf(-t.ch, temp, 1.44269502f) + 1.92596299e-8f, temp) : 0.f;
  t.span = __fdiv_rd(125.49f, t.ch);
  return t;
}

__device__ __forceinline__ Scale make_scale(float zmax, const Rate& t, bool inf) {
  Scale s;
  s.zmax = zmax;
  s.kmax = okey(zmax + 0.f);
  s.c64 = t.ch * kTab;
  s.cl64 = t.cl * kTab;
  const bool near = fabsf(zmax) * t.ch < 32768.f;
  s.zp = near ? 0.f : zmax;
  const float d = zmax - s.zp, ph = d * s.c64, n0 = rintf(ph);
  s.mu = (ph - n0) + fmaf(d, s.cl64, fmaf(d, s.c64, -ph));
  s.nbias = kMagicBits + static_cast<int>(n0);
  s.zmin = fmaxf(__fadd_ru(zmax, -t.span), -kFltMax);
  s.plain = near && !inf && s.zmin > -kFltMax && (zmax - s.zmin) * t.ch > 100.f;
  return s;
}

// 2^(r/64) - 1 for |r| <= 1/2: powers of ln 2 / 64 over factorials, the next term is below 4e-11
__device__ __forceinline__ float exp_rest(float r, float last) {
  return fmaf(fmaf(fmaf(2.11731752e-7f, r, 5.86490495e-5f), r, 1.08304247e-2f), r, last);
}

// w = wh + wl of a logit: rounding of r 2^-31, of the series 2^-31, of wl 2^-31 (|wl| <= wh / 128): relative
// error under 2^-29. The product is never fused with a later sum, so that a weight is the same wherever
// it is asked for.
__device__ __forceinline__ void weight_plain(float x, const Scale& s, const int2* tab, float& wh, float& wl) {
  const float z = fmaxf(x, s.zmin);
  const float m = fmaf(z, s.c64, kMagic);
  const float r = fmaf(z, s.cl64, fmaf(z, s.c64, -(m - kMagic)));
  const uint32_t n = __float_as_uint(m);
  const int2 t = tab[n & (kTab - 1)];
  wh = __uint_as_float(static_cast<uint32_t>(t.x) + (n << 17));
  wl = __fmul_rn(wh, exp_rest(r, __int_as_float(t.y)));
}

// weight_plain of two logits
__device__ __forceinline__ void weight_plain2(float x0, float x1, const Scale& s, const int2* tab, f32x2& wh, f32x2& wl) {
  const f32x2 z = two(fmaxf(x0, s.zmin), fmaxf(x1, s.zmin)), c = two(s.c64, s.c64), magic = two(kMagic, kMagic);
  const f32x2 m = fma2(z, c, magic);
  const f32x2 r = fma2(z, two(s.cl64, s.cl64), fma2(z, c, fma2(m, two(-1.f, -1.f), magic)));
  float m0, m1;
  apart(m, m0, m1);
  const uint32_t n0 = __float_as_uint(m0), n1 = __float_as_uint(m1);
  const int2 t0 = tab[n0 & (kTab - 1)], t1 = tab[n1 & (kTab - 1)];
  wh = two(__uint_as_float(static_cast<uint32_t>(t0.x) + (n0 << 17)), __uint_as_float(static_cast<uint32_t>(t1.x) + (n1 << 17)));
  f32x2 q = fma2(two(2.11731752e-7f, 2.11731752e-7f), r, two(5.86490495e-5f, 5.86490495e-5f));
  q = fma2(q, r, two(1.08304247e-2f, 1.08304247e-2f));
  wl = mul2(wh, fma2(q, r, two(__int_as_float(t0.y), __int_as_float(t1.y))));
}

// the same for any row: 0 below zmin and for NaN, +inf counts as the largest finite number
__device__ __forceinline__ void weight_any(float x, const Scale& s, const float2* pow, float& wh, float& wl) {
  const float d = fminf(fmaxf(x, s.zmin), kFltMax) - s.zp;
  const float m = fmaf(d, s.c64, kMagic);
  const float r = fmaf(d, s.c64, -(m - kMagic)) + fmaf(d, s.cl64, -s.mu);
  const int n = __float_as_int(m) - s.nbias;
  const float2 t = pow[n & (kTab - 1)];
  wh = x >= s.zmin ? __int_as_float(__float_as_int(t.x) + ((n >> 6) << 23)) : 0.f;
  wl = __fmul_rn(wh, exp_rest(r, t.y));
}

__device__ __forceinline__ void weight(float x, const Scale& s, const int2* tab, const float2* pow, float& wh, float& wl) {
  if (s.plain) weight_plain(x, s, tab, wh, wl);
  else weight_any(x, s, pow, wh, wl);
}

// the row's table of weight_plain, by the first 64 threads: entry i is 2^((i - n0 - mu) / 64)
__device__ __forceinline__ void make_table(const Scale& s, const float2* pow, int2* tab) {
  const int i = threadIdx.x;
  if (i >= kTab || !s.plain) return;
  const int n = i - (s.nbias - kMagicBits);
  const float2 t = pow[n & (kTab - 1)];
  const float e = exp_rest(-s.mu, t.y);
  const float h = fmaf(t.x, e, t.x);
  const float rest = fmaf(t.x, e, t.x - h) / h;
  tab[i] = make_int2(__float_as_int(h) + ((n >> 6) << 23) - (i << 17), __float_as_int(rest));
}

// round(w 2^43) = A 2^22 + B, |B| <= 2^21 + 1: both as the bits of the rounded fp32 numbers, biased
__device__ __forceinline__ void weight_parts(float wh, float wl, uint32_t& a, uint32_t& b) {
  const float fa = fmaf(wh + wl, 2097152.f, kMagic);
  const float lo = fmaf(fa - kMagic, -1.f / 2097152.f, wh) + wl;
  a = __float_as_uint(fa);
  b = __float_as_uint(fmaf(lo, 8796093022208.f, kMagic));
}
__device__ __forceinline__ uint64_t weight_of(uint32_t a, uint32_t b) {
  constexpr uint64_t bias = static_cast<uint64_t>(kMagicBits) * 4194305ull;
  return static_cast<uint64_t>(a) * 4194304ull + b - bias;
}
__device__ __forceinline__ uint64_t weight_int(float wh, float wl) {
  uint32_t a, b;
  weight_parts(wh, wl, a, b);
  return weight_of(a, b);
}

// weight_parts of two
__device__ __forceinline__ void weight_parts2(f32x2 wh, f32x2 wl, uint32_t* a, uint32_t* b) {
  const f32x2 magic = two(kMagic, kMagic);
  const f32x2 fa = fma2(add2(wh, wl), two(2097152.f, 2097152.f), magic);
  const f32x2 lo = add2(fma2(add2(fa, two(-kMagic, -kMagic)), two(-1.f / 2097152.f, -1.f / 2097152.f), wh), wl);
  const f32x2 fb = fma2(lo, two(8796093022208.f, 8796093022208.f), magic);
  a[0] = static_cast<uint32_t>(fa);
  a[1] = static_cast<uint32_t>(fa >> 32);
  b[0] = static_cast<uint32_t>(fb);
  b[1] = static_cast<uint32_t>(fb >> 32);
}

// weights of four neighbours
__device__ __forceinline__ void weights4(const float (&x)[4], const Scale& s, const int2* tab, const float2* pow, f32x2 (&wh)[2], f32x2 (&wl)[2]) {
  if (s.plain) {
    weight_plain2(x[0], x[1], s, tab, wh[0], wl[0]);
    weight_plain2(x[2], x[3], s, tab, wh[1], wl[1]);
  } else {
    float h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) weight_any(x[e], s, pow, h[e], l[e]);
    wh[0] = two(h[0], h[1]);
    wh[1] = two(h[2], h[3]);
    wl[0] = two(l[0], l[1]);
    wl[1] = two(l[2], l[3]);
  }
}

// S * f for f in [0, 1), rounded down or up
__device__ __forceinline__ uint64_t mul_fraction(uint64_t S, float f, bool up) {
  const uint32_t b = __float_as_uint(f);
  int e = static_cast<int>(b >> 23);
  uint64_t m = b & 0x7fffffu;
  if (e > 0) m |= 0x800000u; else e = 1;
  const int q = 150 - e;                                     // f = m 2^-q, q >= 24
  if (m == 0) return 0;
  if (q >= 100) return up ? 1 : 0;                           // S m < 2^88
  unsigned __int128 x = static_cast<unsigned __int128>(S) * m;
  if (up) x += (static_cast<unsigned __int128>(1) << q) - 1;
  return static_cast<uint64_t>(x >> q);
}

__device__ __forceinline__ uint32_t cluster_nctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}

// vector v of the row that starts `off` elements behind `base`: what reaches beyond its V elements is -inf
template <typename T>
__device__ __noinline__ uint4 edge(const uint8_t* base, int off, int V, int v) {
  constexpr int VE = 16 / sizeof(T);
  const T* p = reinterpret_cast<const T*>(base) + static_cast<int64_t>(v) * VE;
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const int i = v * VE + e - off;
    const bool ok = i >= 0 && i < V;
    if constexpr (sizeof(T) == 4) {
      w[e] = ok ? __float_as_uint(p[e]) : 0xff800000u;
    } else {
      const uint32_t h = ok ? p[e] : 0xff80u;
      w[e >> 1] |= (e & 1) ? h << 16 : h;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// RES: all of the row's vectors are in shared memory
template <typename T, bool RES>
struct Row {
  static constexpr int VE = 16 / sizeof(T);
  const uint8_t* base;                     // 16-byte aligned, at or before the row's first element
  int off;                                 // elements between the two
  int V;
  uint4* data;                             // this CTA's vectors, [warp][nres]
  const uint4* ends;                       // in shared memory, where vectors are read from L2
  int nres, nvw, nvec;                     // vectors of a warp in shared memory, of a warp, of the row
  int v0, nw;                              // this warp's first vector and their number

  __device__ __forceinline__ static float elem(const uint4& q, int e) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
  }
  __device__ __forceinline__ bool inside(int v) const { return v * VE - off >= 0 && (v + 1) * VE - off <= V; }
  // vector k of warp `w`, whose first vector is `first`; ends: the row's first and last vector
  __device__ __forceinline__ uint4 get(int w, int first, int k) const {
    if (RES || k < nres) return data[w * nres + k];
    const int v = first + k;
    return inside(v) ? __ldg(reinterpret_cast<const uint4*>(base) + v) : ends[v == 0 ? 0 : 1];
  }
  // f(four neighbours as they stand in the row, the first one's index) for every four of this warp
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int k = lane; k < nw; k += 32) {
      const uint4 q = get(w, v0, k);
      const int i = (v0 + k) * VE - off;
#pragma unroll
      for (int g = 0; g < VE; g += 4) {
        const float x[4] = {elem(q, g), elem(q, g + 1), elem(q, g + 2), elem(q, g + 3)};
        f(x, i + g);
      }
    }
  }
};

// exclusive sum over the CTA's threads, *total the whole; `part` holds a number a warp
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* part, uint64_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                         // `part` may still be read from the call before
  if (lane == 31) part[wid] = x;
  __syncthreads();
  uint64_t w = lane < kWarps ? part[lane] : 0;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, kWarps - 1);
  const uint64_t before = __shfl_sync(0xffffffffu, w, max(wid - 1, 0));
  return x - v + (wid > 0 ? before : 0);
}

// sum over the cluster of one number a thread; *before that of the CTAs of lower rank, *mine this
// CTA's, sh.wsum its warps'. Slot `ex` is written once.
__device__ __forceinline__ uint64_t cluster_sum(uint64_t v, Shared& sh, int ex, int rank, int C, uint64_t* before, uint64_t* mine) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  v = warp_sum(v);
  if (lane == 0) sh.wsum[wid] = v;
  __syncthreads();
  if (tid < C) {
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sh.wsum[w];
    *peer(&sh.ex_sum[ex][rank], tid) = t;
  }
  cluster_sync();
  uint64_t total = 0;
  *before = 0;
  *mine = sh.ex_sum[ex][rank];
  for (int c = 0; c < C; ++c) {
    if (c == rank) *before = total;
    total += sh.ex_sum[ex][c];
  }
  return total;
}

template <int BINS>
__device__ __forceinline__ void clear_bins(Shared& sh, int buf) {
  for (int i = threadIdx.x; i < BINS; i += kThreads) sh.hist[buf][0][i] = sh.hist[buf][1][i] = sh.hist[buf][2][i] = sh.hist[buf][3][i] = 0u;
  if (threadIdx.x == 0) sh.sel_bin = 0;
  __syncthreads();
}

// add one token to a bin. SMALL: of at most 2^16 a CTA, so that the sums of the weight's three parts fit a
// word each and no addition has to wait for a carry (the last one is rare); else the low word's carry goes
// into the high one, whose sum over 2^20 tokens is at most 2^31
template <bool COUNT, bool SMALL>
__device__ __forceinline__ void add_to_bin(Shared& sh, int buf, int bin, uint64_t W) {
  if (COUNT) atomicAdd(&sh.hist[buf][0][bin], 1u);
  const uint32_t l = static_cast<uint32_t>(W);
  uint32_t h = static_cast<uint32_t>(W >> 32);
  if (SMALL) {
    atomicAdd(&sh.hist[buf][1][bin], l & 0xffffu);
    atomicAdd(&sh.hist[buf][2][bin], l >> 16);
  } else {
    h += atomicAdd(&sh.hist[buf][1][bin], l) > ~l ? 1u : 0u;
  }
  if (h != 0) atomicAdd(&sh.hist[buf][3][bin], h);
}

// The last bin that is not empty and before which the target is not reached (n0, e0: what lies
// before the first bin); every CTA finds the same. A bin of tokens without weight counts as
// empty where weights are asked for: no target above the weight before them is left there.
template <bool COUNT, int BINS>
__device__ int find_bin(Shared& sh, int buf, int C, uint64_t target, uint64_t& n0, uint64_t& e0, uint64_t* incl, uint64_t* count) {
  const int tid = threadIdx.x;
  uint64_t n[2] = {0, 0}, w[2] = {0, 0};
  for (int c = 0; c < C && 2 * tid < BINS; ++c) {
    const uint2 b = reinterpret_cast<const uint2*>(peer(sh.hist[buf][1], c))[tid];
    const uint2 d = reinterpret_cast<const uint2*>(peer(sh.hist[buf][2], c))[tid];
    const uint2 g = reinterpret_cast<const uint2*>(peer(sh.hist[buf][3], c))[tid];
    w[0] += (static_cast<uint64_t>(g.x) << 32) + (static_cast<uint64_t>(d.x) << 16) + b.x;
    w[1] += (static_cast<uint64_t>(g.y) << 32) + (static_cast<uint64_t>(d.y) << 16) + b.y;
    if (COUNT) {
      const uint2 a = reinterpret_cast<const uint2*>(peer(sh.hist[buf][0], c))[tid];
      n[0] += a.x;
      n[1] += a.y;
    }
  }
  uint64_t total;
  const uint64_t eb = e0 + block_scan(w[0] + w[1], sh.part, &total);
  const uint64_t nb = COUNT ? n0 + block_scan(n[0] + n[1], sh.part2, &total) : 0;
  const uint64_t ee[2] = {eb, eb + w[0]}, nn[2] = {nb, nb + n[0]};
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (COUNT ? (n[j] > 0 && nn[j] < target) : (w[j] > 0 && ee[j] < target)) atomicMax(&sh.sel_bin, static_cast<uint32_t>(2 * tid + j));
  __syncthreads();
  const int bin = static_cast<int>(sh.sel_bin);
  if (bin >> 1 == tid) {
    const bool odd = bin & 1;
    sh.sel_e = odd ? ee[1] : ee[0];
    sh.sel_incl = odd ? ee[1] + w[1] : ee[1];
    sh.sel_n = static_cast<uint32_t>(odd ? nn[1] : nn[0]);
    sh.sel_cnt = static_cast<uint32_t>(odd ? n[1] : n[0]);
  }
  __syncthreads();
  n0 = sh.sel_n;
  e0 = sh.sel_e;
  *incl = sh.sel_incl;
  *count = sh.sel_cnt;
  return bin;
}

__device__ __forceinline__ uint64_t comp_of(float z, int i, uint32_t kmax) {
  return (static_cast<uint64_t>(kmax - okey(z + 0.f)) << kIdxBits) + static_cast<uint32_t>(i);
}

// Tokens near a border: those x >= cut (`per` == 0), or those of one bin of values of them. `maybe` is
// true for all of them and few others, in two instructions.
struct Pick {
  float cut, top, per, mid, half;
  int bin;
  __device__ __forceinline__ int bin_of(float x) const { return __float_as_int(fmaf(top - fminf(x, kFltMax), per, kMagic)) - kMagicBits; }
  __device__ __forceinline__ bool maybe(float x) const { return fabsf(x - mid) <= half; }
  __device__ __forceinline__ bool operator()(float x) const { return x >= cut && (per == 0.f || bin_of(x) == bin); }
};

// bins of the values from `cut` up to the row's largest: rounded, but never falling as the value falls
__device__ __forceinline__ Pick bins_from(const Scale& sc, float cut) {
  const float range = sc.zmax - cut, per = range > 0.f ? __fdiv_rd(kLin - 2.f, range) : 0.f;
  return {cut, sc.zmax, per < kFltMax ? per : 0.f, 0.f, INFINITY, 0};
}
// `maybe` of the one bin chosen
__device__ __forceinline__ void narrow(Pick& pick, const Scale& sc) {
  if (!sc.plain) return;
  const float range = sc.zmax - pick.cut, width = range * (1.f / (kLin - 2));
  pick.mid = fmaf(-width, static_cast<float>(pick.bin), sc.zmax);
  pick.half = fmaf(fabsf(sc.zmax) + range, 1e-6f, 0.501f * width) + 1.17549435e-38f;
}

// The bound of comp below which the tokens stay, COUNT: the first `target` of them, else those before
// which the weight is below `target` (> 0). Looked at: the tokens of `pick`, before which lies the
// weight e0. Returns the bound and the weight of those that stay. One level for each 9 bits of comp.
// The way for rows whose border has more tokens than a list holds. (Out of line, what it needs of
// the caller in shared memory: the caller's registers stay its own.)
template <bool COUNT, typename T, bool RES>
__device__ __noinline__ ulonglong2 select(const Row<T, RES>* shared_row, const Scale* shared_scale, const Pick* shared_pick, uint64_t target,
                                          uint64_t e0, Shared& sh, int C) {
  uint64_t n0 = 0, count, lo = 0, kept;
  int buf = 0, width = 32 + kIdxBits;
  cluster_sync();                          // another CTA may still read the bins or the list of before
  Row<T, RES> row = *shared_row;
  const int wid = threadIdx.x >> 5;
  row.v0 += wid * row.nvw;                 // the row there is that of the first warp
  row.nw = max(0, min(row.nvw, row.nvec - row.v0));
  const Scale sc = *shared_scale;
  const Pick pick = *shared_pick;
  for (;;) {
    const int shift = max(0, width - kBinBits);
    clear_bins<kBins>(sh, buf);
    row.each([&](const float (&x)[4], int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!pick(x[e])) continue;
        const uint64_t at = comp_of(fminf(x[e], kFltMax), i + e, sc.kmax) - lo;       // wraps to a large number below lo
        if (at >> width != 0) continue;
        float wh, wl;
        weight(x[e], sc, sh.tab, sh.pow, wh, wl);
        add_to_bin<true, RES>(sh, buf, static_cast<int>(at >> shift), weight_int(wh, wl));
      }
    });
    cluster_sync();
    const int bin = find_bin<COUNT, kBins>(sh, buf, C, target, n0, e0, &kept, &count);
    buf ^= 1;
    lo += static_cast<uint64_t>(bin) << shift;
    if (shift == 0 || (COUNT && n0 + count <= target)) return make_ulonglong2(lo + (1ull << shift), kept);
    width = shift;
  }
}

// Sort the first P (a power of two up to kMerged) entries of `list` ascending, a bitonic network: thread t
// holds entries E t .. E t + E - 1 in registers (P <= E kThreads), neighbours up to 32 E apart meet by shuffles
// and only wider steps pass through shared memory. 2048 entries take about 7000 clocks of a CTA, 512
// about 4000 (with every step wider than 32 through shared memory the 2048 took 40000).
template <int E>
__device__ __forceinline__ void sort_entries(uint64_t* list, int P) {
  const int tid = threadIdx.x, i0 = tid * E;
  uint64_t v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = i0 + e < P ? list[i0 + e] : kAll;
  auto pick = [](uint64_t a, uint64_t b, bool low) { return (b < a) == low ? b : a; };
  for (int k = 2; k <= P; k <<= 1) {
    for (int j = k >> 1; j >= 32 * E; j >>= 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (i0 + e < P) list[i0 + e] = v[e];
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (i0 + e < P) v[e] = pick(v[e], list[(i0 + e) ^ j], (((i0 + e) & k) == 0) == (((i0 + e) & j) == 0));
    }
#pragma unroll
    for (int j = 16 * E; j >= E; j >>= 1) {
      if (j >= k) continue;
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[e] = pick(v[e], __shfl_xor_sync(0xffffffffu, v[e], j / E), (((i0 + e) & k) == 0) == (((i0 + e) & j) == 0));
    }
#pragma unroll
    for (int j = E >> 1; j > 0; j >>= 1) {
      if (j >= k) continue;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((e & j) == 0) {
          const uint64_t a = v[e], b = v[e | j];
          const bool up = ((i0 + e) & k) == 0;
          v[e] = pick(a, b, up);
          v[e | j] = pick(a, b, !up);
        }
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (i0 + e < P) list[i0 + e] = v[e];
  __syncthreads();
}
__device__ __noinline__ void sort_list(uint64_t* list, int P) {
  if (P <= kThreads) sort_entries<1>(list, P);
  else if (P <= 2 * kThreads) sort_entries<2>(list, P);
  else sort_entries<4>(list, P);
}

__device__ __forceinline__ int padded(int n) {
  int P = 32;
  while (P < n) P <<= 1;
  return P;
}

// The sorted tokens of all CTAs' lists in every CTA's sh.sorted: each CTA sorts its own, finds how many of
// each other's lie before each of its tokens, all lists in step, and puts the token there in every CTA.
// 1400 tokens of four CTAs take 20000 to 35000 clocks; all sorted in each CTA they took 35000 to 55000.
__device__ __noinline__ void merge_lists(Shared& sh, int C, int rank) {
  const int tid = threadIdx.x, own = static_cast<int>(sh.list_n), P = padded(own);
  for (int i = own + tid; i < P; i += kThreads) sh.list[i] = kAll;
  __syncthreads();
  sort_list(sh.list, P);
  cluster_sync();
  int n[kMaxCluster];
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) n[c] = c < C && c != rank ? static_cast<int>(*peer(&sh.list_n, c)) : 0;
  for (int i = tid; i < own; i += kThreads) {
    const uint64_t comp = sh.list[i];
    int at[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) at[c] = 0;
#pragma unroll 1
    for (int step = kList; step > 0; step >>= 1)
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (at[c] + step <= n[c] && peer(sh.list, c)[at[c] + step - 1] < comp) at[c] += step;
    int to = i;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) to += at[c];
    for (int c = 0; c < C; ++c) peer(sh.sorted, c)[to] = comp;
  }
  cluster_sync();
}

// The tokens of `pick` (one at least), as comp, of all CTAs in sh.sorted; returns their number, or -1 where they are too many. Every
// CTA gets the same.
template <typename R>
__device__ __forceinline__ int gather(const R& row, const Scale& sc, Shared& sh, int C, const Pick& pick) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  row.each([&](const float (&x)[4], int i) {
    if (!(pick.maybe(x[0]) || pick.maybe(x[1]) || pick.maybe(x[2]) || pick.maybe(x[3]))) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (pick(x[e])) {
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kList) sh.list[at] = comp_of(fminf(x[e], kFltMax), i + e, sc.kmax);
      }
  });
  cluster_sync();
  // one warp a CTA of the cluster; every warp knows all counts
  uint32_t k = lane < C ? *peer(&sh.list_n, lane) : 0;
  const bool fits = __all_sync(0xffffffffu, k <= kList);
  uint32_t before = 0, n = 0;
  for (int c = 0; c < C; ++c) {
    const uint32_t kc = __shfl_sync(0xffffffffu, k, c);
    if (c < wid) before += kc;
    n += kc;
  }
  if (!fits || n > kMerged) return -1;
  if (n > 2 * kThreads) {
    merge_lists(sh, C, static_cast<int>(cluster_rank()));
    return static_cast<int>(n);
  }
  k = __shfl_sync(0xffffffffu, k, wid & (kMaxCluster - 1));
  const int P = padded(static_cast<int>(n));
  if (wid < C) {
    const uint64_t* from = peer(sh.list, wid);
    for (uint32_t i = lane; i < k; i += 32) sh.sorted[before + i] = from[i];
  } else if (wid >= kMaxCluster) {
    for (int i = static_cast<int>(n) + tid - 32 * kMaxCluster; i < P; i += kThreads - 32 * kMaxCluster) sh.sorted[i] = kAll;
  }
  __syncthreads();
  sort_list(sh.sorted, P);
  return static_cast<int>(n);
}

// Of the n tokens in sh.sorted, before which lies the weight e0: those that stay, in their order,
// under `k` tokens, the sum before a token below ceil(top_p * sum of the first k) (or below
// `target`, where that is not 0) and min-p. *kept: e0 and their weight. At least one stays.
__device__ int cut_sorted(Shared& sh, const Scale& sc, int n, uint64_t e0, int k, float top_p, uint64_t target, float min_p, uint64_t* kept) {
  const int tid = threadIdx.x;
  const int per = (n + kThreads - 1) / kThreads;             // up to 4 neighbours a thread
  uint64_t W[kMerged / kThreads], own = 0, total;
  bool mp[kMerged / kThreads];
  n = min(n, k);
#pragma unroll
  for (int e = 0; e < kMerged / kThreads; ++e) {
    const int j = tid * per + e;
    W[e] = 0;
    mp[e] = true;
    if (e < per && j < n) {
      const float z = okey_value(sc.kmax - static_cast<uint32_t>(sh.sorted[j] >> kIdxBits));
      float wh, wl;
      weight(z, sc, sh.tab, sh.pow, wh, wl);
      W[e] = weight_int(wh, wl);
      mp[e] = !(min_p > 0.f) || z >= sc.zmax || (wh - min_p) + wl >= 0.f;
    }
    own += W[e];
  }
  const uint64_t before = block_scan(own, sh.part, &total);
  if (target == 0) target = top_p < 1.f ? max(mul_fraction(total, fmaxf(top_p, 0.f), true), uint64_t{1}) : kAll;
  uint64_t b = e0 + before, mine = 0;
  int stay = 0;
#pragma unroll
  for (int e = 0; e < kMerged / kThreads; ++e) {
    const int j = tid * per + e;
    if (e < per && j < n && (j == 0 || (b < target && mp[e]))) {
      ++stay;
      mine += W[e];
    }
    b += W[e];
  }
  mine = warp_sum(mine);
  stay = __reduce_add_sync(0xffffffffu, stay);
  if ((tid & 31) == 0) {
    sh.part2[tid >> 5] = mine;
    sh.wkey[tid >> 5] = static_cast<uint32_t>(stay);
  }
  __syncthreads();
  uint64_t sum = 0;
  int m = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    sum += sh.part2[w];
    m += static_cast<int>(sh.wkey[w]);
  }
  *kept = e0 + sum;
  return m;
}

// grid (rows * C), clusters of C CTAs: one row each
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads, 2) k_sample(Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  using R = Row<T, RES>;
  constexpr int VE = R::VE;
  __shared__ R shared_row;
  __shared__ Scale shared_scale;
  __shared__ Pick shared_pick;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int C = static_cast<int>(cluster_nctas());
  const int rank = static_cast<int>(cluster_rank());
  const int64_t r = blockIdx.x / C;
  const int64_t set = r / p.rows_per;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.blk_len != nullptr) {
    // rows of tokens that are not there stay as they were: row 1 + k Dmax + d - 1 needs d <= blk_len[k]
    const int64_t n = static_cast<int64_t>(p.NB) * p.Dmax;
    const int64_t b = r / (1 + n), t = r % (1 + n) - 1;
    if (t >= 0 && t % p.Dmax >= __ldg(p.blk_len + b * p.NB + t / p.Dmax)) return;
  }
  // this CTA runs: the others of the cluster may write to its shared memory (they wait for that before they do)
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const uint8_t* start = static_cast<const uint8_t*>(p.logits) + r * p.row_bytes;
  R row;
  row.off = static_cast<int>((reinterpret_cast<uintptr_t>(start) & 15) / sizeof(T));
  row.base = start - row.off * sizeof(T);
  row.V = p.V;
  row.nres = p.nres;
  row.data = reinterpret_cast<uint4*>(smem);
  row.ends = sh.ends;
  const int nvec = (row.off + p.V + VE - 1) / VE;
  row.v0 = (rank * kWarps + wid) * p.nvw;
  row.nw = max(0, min(p.nvw, nvec - row.v0));
  row.nvw = p.nvw;
  row.nvec = nvec;

  // every vector of this thread is on its way at once
  for (int k = lane; k < min(row.nw, row.nres); k += 32) {
    uint4* dst = row.data + wid * row.nres + k;
    const int v = row.v0 + k;
    if (row.inside(v))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)),
                   "l"(reinterpret_cast<const uint4*>(row.base) + v)
                   : "memory");
    else
      *dst = edge<T>(row.base, row.off, p.V, v);
  }
  if (!RES && tid < 2) sh.ends[tid] = edge<T>(row.base, row.off, p.V, tid == 0 ? 0 : nvec - 1);
  if (tid < kTab) sh.pow[tid] = kPowers.v[tid];
  float temp = p.temperature != nullptr ? __ldg(p.temperature + set) : 1.f;
  int64_t k = p.top_k != nullptr ? __ldg(p.top_k + set) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + set) : 1.f;
  float min_p = p.min_p != nullptr ? __ldg(p.min_p + set) : 0.f;
  if (!(temp >= 0.f)) {
    if (tid == 0) record_error(p.hdr, SSD_ERR_DEVICE, 501);
    temp = 0.f;
  }
  if (temp == 0.f) {                       // greedy: the first of the largest
    temp = 1.f;
    k = 1;
  }
  temp = fminf(fmaxf(temp, 0x1.715476p-120f), 0x1p100f);     // from log2(e) 2^-120, whose rate is 2^120, on
  min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;             // NaN: all
  if (k < 0 || k >= p.V) k = 0;
  const Rate rate = make_rate(temp);
  // how far below the largest a token may lie whose weight is (1 - top_p) / V of it
  const float depth = top_p < 1.f ? __fmul_ru(-logf((1.f - fmaxf(top_p, 0.f)) / static_cast<float>(p.V) * 0.999f), temp) : 0.f;
  // with top-k: the tokens that each CTA that holds any answers for. A value that many of its tokens reach is
  // found, and the least of these values is reached by k tokens of the row
  const int warps = (nvec + p.nvw - 1) / p.nvw, ctas = (warps + kWarps - 1) / kWarps;
  const int share = static_cast<int>((k + ctas - 1) / ctas);
  if (tid == 0) sh.list_n = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!RES) __syncthreads();               // the ends

  // ---- the row's largest value; with top-k also a value that k tokens at least reach
  float mx = -INFINITY;
  row.each([&](const float (&x)[4], int) { mx = fmaxf(fmaxf(mx, fmaxf(x[0], x[1])), fmaxf(x[2], x[3])); });
  uint32_t reach = 0;                      // as okey; 0: none found
  const uint32_t key = okey(fminf(mx, kFltMax) + 0.f);
  const bool few = k > 0 && share <= kWarps * kTop / 2;
  if (few) {
    uint32_t left = key;
#pragma unroll
    for (int j = 0; j < kTop; ++j) {
      const uint32_t most = __reduce_max_sync(0xffffffffu, left);
      const uint32_t who = __ballot_sync(0xffffffffu, left == most);
      if (lane == __ffs(who) - 1) left = 0;
      if (lane == 0) sh.wkey[wid * kTop + j] = row.nw > 0 ? most : 0;
    }
  }
  {
    const float m = warp_max(mx);
    if (lane == 0) sh.wmax[wid] = m;
  }
  __syncthreads();
  if (few) {
    // the share-th largest of the warps' kTop largest each: the largest that as many reach
    if (wid == 0) {
#pragma unroll
      for (int j = 0; j < kWarps * kTop / 32; ++j) {
        const uint32_t v = sh.wkey[32 * j + lane];
        int n = 0;
        for (int i = 0; i < kWarps * kTop; ++i) n += sh.wkey[i] >= v ? 1 : 0;
        reach = max(reach, __reduce_max_sync(0xffffffffu, n >= share ? v : 0u));
      }
    }
  } else if (k > 0 && share <= 2 * kThreads) {
    // the share-th largest of the threads' largest (with more tokens than threads: half the share by
    // their second largest, which two tokens reach), to 16 bits
    uint32_t own = key;
    int want = share;
    if (share > kThreads) {
      float m1 = -INFINITY, m2 = -INFINITY;
      row.each([&](const float (&x)[4], int) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m2 = fmaxf(m2, fminf(m1, x[e] > -INFINITY ? x[e] : -INFINITY));
          m1 = fmaxf(m1, x[e]);
        }
      });
      own = okey(fminf(m2, kFltMax) + 0.f);
      want = (share + 1) / 2;
    }
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t t = reach | (1u << bit);
      if (__syncthreads_count(own >= t) >= want) reach = t;
    }
  }
  if (rank >= ctas) reach = ~0u;           // a CTA without tokens does not count
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (tid < C) {
    float t = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t = fmaxf(t, sh.wmax[w]);
    *peer(&sh.ex_max[rank], tid) = t;
    *peer(&sh.ex_key[rank], tid) = reach;
  }
  cluster_sync();
  float zmax = -INFINITY;
  reach = ~0u;
  for (int c = 0; c < C; ++c) {
    zmax = fmaxf(zmax, sh.ex_max[c]);
    reach = min(reach, sh.ex_key[c]);
  }
  const bool empty = !(zmax > -INFINITY);
  const Scale sc = make_scale(fminf(zmax, kFltMax), rate, zmax == INFINITY);
  make_table(sc, sh.pow, sh.tab);
  if (tid == 0) {
    shared_row = row;
    shared_scale = sc;
  }
  __syncthreads();

  uint64_t bound = kAll, S = 0, before = 0, mine = 0;
  int stays = 0;
  bool known = false, all_cut = false;       // S is that of the tokens that stay; min-p is in the bound
  if (!empty) {
    if (k > 0) {
      const float low = reach > okey(-INFINITY) ? okey_value(reach) : -kFltMax;
      // from low to zmax, a little wider; of rows that are not plain every number: there may be infinities
      const float span = 0.5f * sc.zmax - 0.5f * low;
      const Pick pick = {low, 0.f, 0.f, sc.plain ? low + span : 0.f,
                         sc.plain ? fmaf(fabsf(sc.zmax) + fabsf(low), 1e-6f, span) + 1.17549435e-38f : INFINITY, 0};
      int n = -1;
      if (k <= kShortK) {
        n = gather(row, sc, sh, C, pick);
        if (n >= 0) {
          const int m = cut_sorted(sh, sc, n, 0, static_cast<int>(k), top_p, 0, min_p, &S);
          bound = sh.sorted[m - 1] + 1;
          stays = m;
          all_cut = true;
        }
      }
      const float range = sc.zmax - low;
      if (n < 0 && low > -kFltMax && range > 1e-30f && range < kFltMax) {
        // many: bins of the values from low up, then the tokens of the bin in which the k-th lies
        if (k <= kShortK) {                // another CTA may still read the list of before
          cluster_sync();
          if (tid == 0) sh.list_n = 0;
        }
        Pick bin = bins_from(sc, low);
        clear_bins<kLin>(sh, 0);
        row.each([&](const float (&x)[4], int) {
          if (!(x[0] >= low || x[1] >= low || x[2] >= low || x[3] >= low)) return;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[e] >= low) {
              float wh, wl;
              weight(x[e], sc, sh.tab, sh.pow, wh, wl);
              add_to_bin<true, RES>(sh, 0, bin.bin_of(x[e]), weight_int(wh, wl));
            }
        });
        cluster_sync();
        uint64_t n0 = 0, e0 = 0, incl, cnt;
        bin.bin = find_bin<true, kLin>(sh, 0, C, static_cast<uint64_t>(k), n0, e0, &incl, &cnt);
        narrow(bin, sc);
        n = gather(row, sc, sh, C, bin);
        if (n >= 0) {
          const int m = cut_sorted(sh, sc, n, e0, static_cast<int>(k - static_cast<int64_t>(n0)), 1.f, kAll, 0.f, &S);
          bound = sh.sorted[m - 1] + 1;
        }
      }
      if (n < 0) {
        if (tid == 0) shared_pick = pick;
        const ulonglong2 got = select<true>(&shared_row, &shared_scale, &shared_pick, static_cast<uint64_t>(k), 0, sh, C);
        bound = got.x;
        S = got.y;
      }
      known = true;
    }
    if (top_p < 1.f && !all_cut) {
      // tokens of a weight below (1 - top_p) / V, together, are not more than the tail that is cut
      // (the sum is at least 1); binned by their value are the others, and all are summed
      const float z_cut = fmaxf(__fadd_rd(sc.zmax, -depth), sc.zmin);
      Pick pick = bins_from(sc, z_cut);
      if (known) {                         // another CTA may still read the bins or the list of before
        cluster_sync();
        if (tid == 0) sh.list_n = 0;
      }
      clear_bins<kLin>(sh, 0);
      uint32_t sa = 0, sb = 0, count = 0;
      row.each([&](const float (&x)[4], int) {
        // (the sum of the first k is known: only the bins are asked for)
        if (known && !(x[0] >= z_cut || x[1] >= z_cut || x[2] >= z_cut || x[3] >= z_cut)) return;
        uint32_t a[4], b[4];
        f32x2 wh[2], wl[2];
        weights4(x, sc, sh.tab, sh.pow, wh, wl);
        weight_parts2(wh[0], wl[0], a, b);
        weight_parts2(wh[1], wl[1], a + 2, b + 2);
        sa += (a[0] + a[1]) + (a[2] + a[3]);
        sb += (b[0] + b[1]) + (b[2] + b[3]);
        count += 4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x[e] >= z_cut) add_to_bin<false, RES>(sh, 0, pick.bin_of(x[e]), weight_of(a[e], b[e]));
      });
      // the biases go out modulo 2^32: a thread holds at most kThreadTokens, so the sums (2^21 each) fit
      sa -= count * kMagicBits;
      sb -= count * kMagicBits;
      const uint64_t sum = cluster_sum(static_cast<uint64_t>(static_cast<int64_t>(static_cast<int>(sa)) * 4194304 + static_cast<int>(sb)), sh, 0, rank, C, &before, &mine);
      const uint64_t target = max(mul_fraction(known ? S : sum, fmaxf(top_p, 0.f), true), uint64_t{1});
      uint64_t n0 = 0, e0 = 0, incl, cnt;
      pick.bin = find_bin<false, kLin>(sh, 0, C, target, n0, e0, &incl, &cnt);
      narrow(pick, sc);
      const int n = gather(row, sc, sh, C, pick);
      if (n >= 0) {
        const int m = cut_sorted(sh, sc, n, e0, n, 1.f, target, 0.f, &S);
        bound = sh.sorted[m - 1] + 1;
      } else {
        if (tid == 0) shared_pick = pick;
        const ulonglong2 got = select<false>(&shared_row, &shared_scale, &shared_pick, target, e0, sh, C);
        bound = got.x;
        S = got.y;
      }
      known = true;
    }
  }
  // kept: z > zt, or z == zt and index < it; none below zmin
  float zt = -INFINITY;
  int it = 0;
  if (bound != kAll) {
    const uint64_t kd = bound >> kIdxBits;
    if (kd < sc.kmax - okey(-INFINITY)) {
      const uint32_t key = sc.kmax - static_cast<uint32_t>(kd);
      it = static_cast<int>(bound & ((1u << kIdxBits) - 1));
      // the key of -0, which no element has, as a bound means all zeros
      if (key == 0x7fffffffu) it = p.V;
      zt = okey_value(key) + 0.f;
    }
  }
  if (zt < sc.zmin) {
    zt = sc.zmin;
    it = p.V;
  }
  const bool use_min_p = min_p > 0.f && !all_cut;
  // the weights of four neighbours and which of them stay; false where none does
  auto kept_weights = [&](const float (&x)[4], int i, f32x2 (&wh)[2], f32x2 (&wl)[2], bool (&stay)[4]) {
    if (!(x[0] >= zt || x[1] >= zt || x[2] >= zt || x[3] >= zt)) return false;
    weights4(x, sc, sh.tab, sh.pow, wh, wl);
#pragma unroll
    for (int e = 0; e < 4; ++e) stay[e] = x[e] > zt;
    if (x[0] == zt || x[1] == zt || x[2] == zt || x[3] == zt || !sc.plain) {
#pragma unroll
      for (int e = 0; e < 4; ++e) stay[e] = x[e] >= zt && (fminf(x[e], kFltMax) > zt || i + e < it);
    }
    if (use_min_p) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float h[2], l[2];
        apart(wh[e >> 1], h[0], h[1]);
        apart(wl[e >> 1], l[0], l[1]);
        stay[e] = stay[e] && (x[e] >= sc.zmax || (h[e & 1] - min_p) + l[e & 1] >= 0.f);
      }
    }
    return true;
  };
  // as integers, 0 for those that do not stay
  auto kept_ints = [&](const float (&x)[4], int i, uint64_t (&W)[4]) {
    f32x2 wh[2], wl[2];
    bool stay[4];
    W[0] = W[1] = W[2] = W[3] = 0;
    if (!kept_weights(x, i, wh, wl, stay)) return;
    uint32_t a[4], b[4];
    weight_parts2(wh[0], wl[0], a, b);
    weight_parts2(wh[1], wl[1], a + 2, b + 2);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (stay[e]) W[e] = weight_of(a[e], b[e]);
  };

  // a few tokens that stay, known in their order: drawn from there, by the first CTA
  const bool from_list = all_cut && stays <= kFew;
  const bool draw = p.token != nullptr && !empty;
  if (!empty && (use_min_p || !known || (draw && !from_list))) {
    uint64_t t = 0;
    row.each([&](const float (&x)[4], int i) {
      uint64_t W[4];
      kept_ints(x, i, W);
      t += (W[0] + W[1]) + (W[2] + W[3]);
    });
    S = cluster_sum(t, sh, 1, rank, C, &before, &mine);
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");     // nothing of another CTA is read any more
  // 2^43 / S as a pair
  float ih = 0.f, il = 0.f;
  if (S > 0) {
    const float s_h = __ull2float_rn(S), s_l = __ll2float_rn(static_cast<int64_t>(S - __float2ull_rn(s_h)));
    ih = __fdiv_rn(8796093022208.f, s_h);
    il = __fdiv_rn(fmaf(-ih, s_l, fmaf(-ih, s_h, 8796093022208.f)), s_h);
  }
  auto probability = [&](float wh, float wl) { return fmaf(wh, ih, fmaf(wh, il, __fmul_rn(wl, ih))); };

  if (p.probs != nullptr) {
    float* out = p.probs + r * p.V;
    const bool wide = ((reinterpret_cast<uintptr_t>(out) / 4 - row.off) & 3) == 0;
    if (wide) {
      row.each([&](const float (&x)[4], int i) {
        f32x2 wh[2], wl[2];
        bool stay[4];
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (kept_weights(x, i, wh, wl, stay)) {
          const f32x2 h = two(ih, ih), l = two(il, il);
          apart(fma2(wh[0], h, fma2(wh[0], l, mul2(wl[0], h))), v[0], v[1]);
          apart(fma2(wh[1], h, fma2(wh[1], l, mul2(wl[1], h))), v[2], v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = stay[e] ? v[e] : 0.f;
        }
        if (i >= 0 && i + 4 <= p.V && in_range(i + 3, p.V, p.hdr, 510)) {
          *reinterpret_cast<float4*>(out + i) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e >= 0 && i + e < p.V) out[i + e] = v[e];
        }
      });
    } else {
      // rows whose elements lie otherwise in 16 bytes than the output's: four bytes a lane
      const int i0 = row.v0 * VE - row.off;
      for (int j = lane; j < row.nw * VE; j += 32) {
        const int i = i0 + j;
        if (i < 0 || i >= p.V || !in_range(i, p.V, p.hdr, 511)) continue;
        const int kv = j / VE;
        const T* src = RES || kv < row.nres ? reinterpret_cast<const T*>(row.data + wid * row.nres) + j
                                     : reinterpret_cast<const T*>(row.base) + static_cast<int64_t>(row.v0) * VE + j;
        float x;
        if constexpr (sizeof(T) == 4) x = *src; else x = bf16_to_f32(*src);
        const float z = fminf(x, kFltMax);
        float v = 0.f;
        if (x >= zt && (z > zt || i < it)) {
          float wh, wl;
          weight(x, sc, sh.tab, sh.pow, wh, wl);
          if (!use_min_p || x >= sc.zmax || (wh - min_p) + wl >= 0.f) v = probability(wh, wl);
        }
        out[i] = v;
      }
    }
  }

  if (p.token != nullptr && empty && rank == 0 && tid == 0) {
    p.token[r] = -1;
    if (p.prob != nullptr) p.prob[r] = 0.f;
  }
  if (draw) {
    float u = __ldg(p.u + r);
    u = u > 0.f ? fminf(u, 0.99999994f) : 0.f;
    const uint64_t thr = mul_fraction(S, u, false);         // the first token with C_i > thr
    auto found = [&](int i, float wh, float wl) {
      p.token[r] = i;
      if (p.prob != nullptr) p.prob[r] = probability(wh, wl);
    };
    if (from_list) {
      if (rank == 0) {
        // the tokens again, by index: 20 bits of it above 44 of the weight
        const int P = padded(stays);
        uint64_t own = kAll;
        if (tid < stays) {
          const uint64_t comp = sh.sorted[tid];
          float wh, wl;
          weight(okey_value(sc.kmax - static_cast<uint32_t>(comp >> kIdxBits)), sc, sh.tab, sh.pow, wh, wl);
          own = (comp & ((1u << kIdxBits) - 1)) << 44 | weight_int(wh, wl);
        }
        const uint64_t comp = tid < stays ? sh.sorted[tid] : 0;
        __syncthreads();
        if (tid < P) sh.sorted[tid] = own;
        __syncthreads();
        sort_list(sh.sorted, P);
        const uint64_t at = tid < stays ? sh.sorted[tid] : 0, W = at & ((1ull << 44) - 1);
        uint64_t all;
        const uint64_t pre = block_scan(W, sh.part, &all);
        if (thr >= pre && thr < pre + W) sh.sel_bin = static_cast<uint32_t>(at >> 44);
        __syncthreads();
        if (tid < stays && (comp & ((1u << kIdxBits) - 1)) == sh.sel_bin) {
          float wh, wl;
          weight(okey_value(sc.kmax - static_cast<uint32_t>(comp >> kIdxBits)), sc, sh.tab, sh.pow, wh, wl);
          found(static_cast<int>(sh.sel_bin), wh, wl);
        }
      }
    } else if (thr >= before && thr < before + mine) {
      // this CTA holds it: the warp, then the four neighbours, then the token
      uint64_t c0 = before;
      int w = 0;
      while (w < kWarps - 1 && thr >= c0 + sh.wsum[w]) c0 += sh.wsum[w++];
      const int first = (rank * kWarps + w) * p.nvw;
      const int groups = max(0, min(p.nvw, nvec - first)) * (VE / 4);
      for (int k0 = 0; k0 < groups; k0 += kThreads) {
        const int g = k0 + tid;
        const int i = first * VE - row.off + 4 * g;
        uint64_t W[4] = {0, 0, 0, 0}, all;
        float x[4];
        if (g < groups) {
          const uint4 q = row.get(w, first, g / (VE / 4));
          const int e0 = g % (VE / 4) * 4;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = e0 == 0 ? R::elem(q, e) : R::elem(q, (e + 4) % VE);
          kept_ints(x, i, W);
        }
        uint64_t pre = c0 + block_scan(W[0] + W[1] + W[2] + W[3], sh.part, &all);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (thr >= pre && thr < pre + W[e]) {
            float wh, wl;
            weight(x[e], sc, sh.tab, sh.pow, wh, wl);
            found(i + e, wh, wl);
          }
          pre += W[e];
        }
        c0 += all;
        if (thr < c0) break;
      }
    }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

constexpr int kMaxData = 160 * 1024;       // a CTA's part of a row in shared memory, at most
// and no more than the 2^16 tokens whose sums in bins fit (add_to_bin)
template <typename T>
constexpr int max_data() {
  return std::min(kMaxData, 65536 * static_cast<int>(sizeof(T)));
}

template <typename T>
static void shape(int nvec, int C, Params& p) {
  p.nvw = (nvec + kWarps * C - 1) / (kWarps * C);
  p.nres = std::min(p.nvw, max_data<T>() / 16 / kWarps);
}

// CTAs of a row and clusters that run at once, for a row of nvec vectors: asked once for each C and
// 4 KB step of shared memory
template <typename T>
static int active_clusters(int dev, int C, size_t bytes) {
  static std::mutex mu;
  static int16_t known[kMaxDevices][kMaxCluster + 1][kMaxData / 4096 + 1];
  const int step = static_cast<int>((bytes + 4095) / 4096);
  std::lock_guard<std::mutex> lock(mu);
  int16_t& n = known[dev][C][step];
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(step) * 4096;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int got = 0;
    if (cudaOccupancyMaxActiveClusters(&got, k_sample<T, true>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      got = 0;
    }
    n = static_cast<int16_t>(got > 0 ? std::min(got, 32000) : -1);
  }
  return n;
}

template <typename T>
static int launch(const Params& in, int64_t rows, cudaStream_t s) {
  constexpr int VE = Row<T, true>::VE;
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return SSD_ERR_CUDA;
  std::call_once(once[dev], [dev] {
    err[dev] = cudaFuncSetAttribute(k_sample<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxData);
    if (err[dev] == cudaSuccess) err[dev] = cudaFuncSetAttribute(k_sample<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxData);
  });
  if (err[dev] != cudaSuccess) return SSD_ERR_CUDA;
  Params p = in;
  const int nvec = (p.V + 2 * VE - 2) / VE;                  // at most, whatever the row's first element's place
  // CTAs a row: the least of (waves of clusters) x (a fixed part, the cluster's barriers, and the CTA's
  // share of the row), both in tokens: 512 threads pass over 12500 of them in the fixed part's time.
  // us with 1 .. 8 CTAs, top-p 0.95 (* the rule's): a row of 128256 fp32 logits 123 65 43 32 29 28 26 25*; 81 of them 132 137
  // 95 102 93 82* 102 97; 64 rows of 151936 bf16 132 73 92 63* 90 86 86 84; 300 of them 283 283 317 252* 274 296 335 330; 648
  // rows of 32000 113* 132 177 197 258 319 394 377; 40 of them 32 23 21 24 24 25* 40 39
  int C = 0;
  double least = 0.;
  for (int c = 1; c <= kMaxCluster; ++c) {
    shape<T>(nvec, c, p);
    if ((p.nvw + 31) / 32 * VE > kThreadTokens) continue;
    const int active = active_clusters<T>(dev, c, static_cast<size_t>(p.nres) * kWarps * 16);
    if (active < 1) continue;
    double part = static_cast<double>(p.nvw) * kWarps * VE;
    if (p.nvw > p.nres) part += 2. * (p.nvw - p.nres) * kWarps * VE;      // read again from L2 by every pass
    const double cost = static_cast<double>((rows + active - 1) / active) * (12500. + part);
    if (C == 0 || cost < least) {
      C = c;
      least = cost;
    }
  }
  if (C == 0) return SSD_ERR_CUDA;
  shape<T>(nvec, C, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.nres) * kWarps * 16;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  {
    KernelTimer timer(SSD_KERNEL_SAMPLE, s);
    if (cudaLaunchKernelEx(&cfg, p.nvw <= p.nres ? k_sample<T, true> : k_sample<T, false>, p) != cudaSuccess) return SSD_ERR_CUDA;
  }
  count_launch();
  return check_launch();
}

// arguments that both calls have in common
static int check(const ssd_rows_args* a) {
  if (a->dtype != SSD_F32 && a->dtype != SSD_BF16) return SSD_ERR_INVALID;
  if (a->R < 0 || a->V < 1 || a->row_stride < a->V || a->rows_per < 1) return SSD_ERR_INVALID;
  if (a->V > (1 << kIdxBits) || a->R > 0x7fffffffLL / kMaxCluster) return SSD_ERR_UNSUPPORTED;
  if (a->R > 0 && a->row_stride > (1LL << 59) / a->R) return SSD_ERR_UNSUPPORTED;
  if (a->R > 0 && a->logits == nullptr) return SSD_ERR_INVALID;
  const size_t es = a->dtype == SSD_BF16 ? 2 : 4;
  if (!aligned(a->logits, es) || !aligned(a->temperature, 4) || !aligned(a->top_k, 4) || !aligned(a->top_p, 4) || !aligned(a->min_p, 4))
    return SSD_ERR_INVALID;
  return SSD_OK;
}

static Params params(const ssd_rows_args* a, void* ws) {
  Params p = {};
  p.logits = a->logits;
  p.row_bytes = a->row_stride * (a->dtype == SSD_BF16 ? 2 : 4);
  p.V = static_cast<int>(a->V);
  p.rows_per = a->rows_per;
  p.temperature = a->temperature;
  p.top_k = a->top_k;
  p.top_p = a->top_p;
  p.min_p = a->min_p;
  p.hdr = static_cast<WsHeader*>(ws);
  return p;
}

// the bytes that the rows and their settings take
constexpr int kRowSpans = 5;
static void row_spans(const ssd_rows_args* a, Span* s) {
  const int64_t es = a->dtype == SSD_BF16 ? 2 : 4, sets = (a->R + a->rows_per - 1) / a->rows_per;
  s[0] = {a->logits, ((a->R - 1) * a->row_stride + a->V) * es};
  s[1] = {a->temperature, 4 * sets};
  s[2] = {a->top_k, 4 * sets};
  s[3] = {a->top_p, 4 * sets};
  s[4] = {a->min_p, 4 * sets};
}

}  // namespace smp
}  // namespace ssd

extern "C" int ssd_filter_probs(const ssd_rows_args* a, const int32_t* blk_len, int NB, int Dmax, float* probs, void* ws,
                                size_t ws_bytes, void* stream) {
  using namespace ssd;
  if (a == nullptr) return SSD_ERR_INVALID;
  const int rc = smp::check(a);
  if (rc != SSD_OK) return rc;
  int64_t batch = 0;
  if (blk_len != nullptr) {
    if (NB < 1 || Dmax < 1 || a->R % (1 + static_cast<int64_t>(NB) * Dmax) != 0) return SSD_ERR_INVALID;
    batch = a->R / (1 + static_cast<int64_t>(NB) * Dmax);
  }
  if (a->R == 0) return SSD_OK;
  if (probs == nullptr || !aligned(probs, 4) || !aligned(blk_len, 4)) return SSD_ERR_INVALID;
  Span spans[2 + smp::kRowSpans] = {{probs, 4 * a->R * a->V}};
  smp::row_spans(a, spans + 1);
  spans[1 + smp::kRowSpans] = {blk_len, 4 * batch * NB};
  if (overlap(spans, 1, 2 + smp::kRowSpans)) return SSD_ERR_INVALID;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
  smp::Params p = smp::params(a, ws);
  p.blk_len = blk_len;
  p.NB = NB;
  p.Dmax = Dmax;
  p.probs = probs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == SSD_BF16 ? smp::launch<uint16_t>(p, a->R, s) : smp::launch<float>(p, a->R, s);
}

extern "C" int ssd_sample(const ssd_rows_args* a, const float* u, int32_t* token, float* prob, float* probs, void* ws,
                          size_t ws_bytes, void* stream) {
  using namespace ssd;
  if (a == nullptr) return SSD_ERR_INVALID;
  const int rc = smp::check(a);
  if (rc != SSD_OK) return rc;
  if (a->R == 0) return SSD_OK;
  if (u == nullptr || token == nullptr) return SSD_ERR_INVALID;
  if (!aligned(u, 4) || !aligned(token, 4) || !aligned(prob, 4) || !aligned(probs, 4)) return SSD_ERR_INVALID;
  Span spans[4 + smp::kRowSpans] = {{token, 4 * a->R}, {prob, 4 * a->R}, {probs, 4 * a->R * a->V}};
  smp::row_spans(a, spans + 3);
  spans[3 + smp::kRowSpans] = {u, 4 * a->R};
  if (overlap(spans, 3, 4 + smp::kRowSpans)) return SSD_ERR_INVALID;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
  smp::Params p = smp::params(a, ws);
  p.u = u;
  p.token = token;
  p.prob = prob;
  p.probs = probs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->dtype == SSD_BF16 ? smp::launch<uint16_t>(p, a->R, s) : smp::launch<float>(p, a->R, s);
}
