// Sampling distributions of logit rows: temperature, top-k, top-p and min-p, as probability
// rows (ssd_filter_probs) and as tokens drawn by a given uniform number (ssd_sample).
//
// Weights w_i = 2^((z_i - z_max) log2(e) / T) are pairs of fp32 numbers (relative error under
// 2^-29) and, where they are summed, integers round(w_i 2^43): the sums are exact, so neither a
// cut nor a token depends on the order in which threads add. The tokens that stay are the first
// ones in the order (z descending, index ascending), so one composite number
//   comp = (okey(z_max) - okey(z)) * 2^20 + index       (okey: the fp32 order as unsigned integers)
// and one bound say which. A bound is found by histograms of 1024 bins of comp (count and weight
// of each), the next one over the bin in which the count passes top-k or the weight passes
// top_p * sum, down to single tokens; ties at the border are thereby cut by their index.
//
// A cluster of 1 to 8 CTAs holds a row in its shared memory: it is read from HBM once, and the
// passes over it (sum, histograms, output) read shared memory. Partial results cross the
// cluster through distributed shared memory. Rows beyond the cluster's shared memory are
// read again from L2.
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
constexpr int kBins = 1024;
constexpr int kBinBits = 10;
constexpr int kMaxCluster = 8;
constexpr int kIdxBits = 20;               // V <= 2^20: the weight sums then fit 64 bits
constexpr int kTab = 64;
constexpr uint64_t kAll = ~0ull;
constexpr int kList = 1024;                // tokens near a border that one CTA may hold,
constexpr int kMerged = 2048;              // and all CTAs of the cluster together, to be sorted

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
  float2 tab[kTab];                        // 2^(i/64) as fp32, and what that lacks relative to it
  union {
    uint32_t hist[2][3][kBins];            // count, low and high word of the weight; two levels in turns
    uint64_t sort[kMerged];
  };
  uint64_t list[kList];                    // this CTA's tokens near a border
  uint64_t ex_sum[2][kMaxCluster];         // from every CTA of the cluster
  float ex_max[kMaxCluster];
  uint32_t ex_key[kMaxCluster];
  uint64_t part[kWarps], part2[kWarps];
  uint64_t wsum[kWarps];
  float wmax[kWarps];
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

// w = 2^((z - zmax) c), c = ch + cl = log2(e) / T, of z >= zmin (where w >= 2^-125.5). With d = z - zp
// exact and zmax's own d c = M, rounded to n0 / 64 and a rest mu:
//   round(64 d ch) - n0 = n,   (z - zmax) c = n / 64 + r,   r = (d ch - round(64 d ch) / 64) + (d cl - mu)
// zp = 0 unless |M| >= 2^15 (the magic number would lose bits): zp = zmax then, and every z >= zmin
// lies within a factor of two of it, so that d is exact again.
struct Scale {
  float zmax, zmin, zp, c64, ch, cl, mu;
  int nbias;
  uint32_t kmax;
};

// In pairs of fp32 numbers: a division in fp64 by every thread of a CTA takes microseconds here
__device__ __forceinline__ Scale make_scale(float zmax, float temp) {
  Scale s;
  s.zmax = zmax;
  s.kmax = okey(zmax + 0.f);
  s.ch = fminf(__fdiv_rn(1.44269502f, temp), 0x1p120f);
  s.cl = s.ch < 0x1p120f ? __fdiv_rn(fmaf(-s.ch, temp, 1.44269502f) + 1.92596299e-8f, temp) : 0.f;
  s.c64 = s.ch * kTab;
  s.zp = fabsf(zmax) * s.ch < 32768.f ? 0.f : zmax;
  const float d = zmax - s.zp, ph = d * s.ch, n0 = rintf(ph * kTab);
  s.mu = fmaf(n0, -1.f / kTab, ph) + fmaf(d, s.cl, fmaf(d, s.ch, -ph));
  s.nbias = kMagicBits + static_cast<int>(n0);
  s.zmin = fmaxf(__fadd_ru(zmax, -__fdiv_rd(125.49f, s.ch)), -kFltMax);
  return s;
}

// w = wh + wl of a logit x: 0 below zmin and for NaN, +inf counts as the largest finite number.
// Rounding: r 2^-31, its power series 2^-31, wl 2^-31 (|wl| <= wh / 128): relative error under 2^-29
__device__ __forceinline__ void weight(float x, const Scale& s, const float2* tab, float& wh, float& wl) {
  const float d = fminf(fmaxf(x, s.zmin), kFltMax) - s.zp;
  const float m = fmaf(d, s.c64, kMagic);
  const float r = fmaf(d, s.ch, (m - kMagic) * (-1.f / kTab)) + fmaf(d, s.cl, -s.mu);
  const int n = __float_as_int(m) - s.nbias;
  const float2 t = tab[n & (kTab - 1)];
  wh = x >= s.zmin ? __int_as_float(__float_as_int(t.x) + ((n >> 6) << 23)) : 0.f;
  // 2^r - 1 for |r| <= 1/128: powers of ln 2 over factorials, the next term is below 4e-11
  const float q = fmaf(fmaf(0.0555041087f, r, 0.2402265070f), r, 0.6931471806f);
  wl = __fmul_rn(wh, fmaf(q, r, t.y));     // never fused with a later sum: a weight is the same wherever it is asked for
}

// round(w 2^43) = A 2^22 + B, |B| <= 2^21 + 1: both as the bits of the rounded fp32 numbers, biased
__device__ __forceinline__ void weight_parts(float wh, float wl, int& a, int& b) {
  const float fa = fmaf(wh + wl, 2097152.f, kMagic);
  const float lo = fmaf(fa - kMagic, -1.f / 2097152.f, wh) + wl;
  a = __float_as_int(fa);
  b = __float_as_int(fmaf(lo, 8796093022208.f, kMagic));
}
__device__ __forceinline__ uint64_t weight_int(float wh, float wl) {
  int a, b;
  weight_parts(wh, wl, a, b);
  return static_cast<uint64_t>(static_cast<int64_t>(a - kMagicBits) * 4194304 + (b - kMagicBits));
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

template <typename T>
struct Row {
  static constexpr int VE = 16 / sizeof(T);
  const uint8_t* base;                     // 16-byte aligned, at or before the row's first element
  int off;                                 // elements between the two
  int V;
  uint4* data;                             // this CTA's vectors, [warp][nres]
  int nres, v0, nw;                        // this warp's first vector and their number

  __device__ __forceinline__ static float elem(const uint4& q, int e) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
  }
  __device__ __forceinline__ bool inside(int v) const { return v * VE - off >= 0 && (v + 1) * VE - off <= V; }
  // the row's first and last vector may reach beyond it: what does is -inf
  __device__ uint4 edge(int v) const {
    const T* p = reinterpret_cast<const T*>(base) + static_cast<int64_t>(v) * VE;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int i = v * VE + e - off;
      const bool ok = i >= 0 && i < V;
      if constexpr (sizeof(T) == 4) {
        w[e] = ok ? __float_as_uint(p[e]) : 0xff800000u;
      } else {
        const uint32_t h = ok ? p[e] : 0xff80u;
        if (e & 1) w[e >> 1] |= h << 16; else w[e >> 1] = h;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 global(int v) const {
    return inside(v) ? __ldg(reinterpret_cast<const uint4*>(base) + v) : edge(v);
  }
  // vector k of warp `w`, whose first vector is `first`
  __device__ __forceinline__ uint4 get(int w, int first, int k) const {
    return k < nres ? data[w * nres + k] : global(first + k);
  }
  // f(value, index) for every element of this warp, as it stands in the row
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int k = lane; k < nw; k += 32) {
      const uint4 q = get(w, v0, k);
      const int i = (v0 + k) * VE - off;
#pragma unroll
      for (int e = 0; e < VE; ++e) f(elem(q, e), i + e);
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

__device__ __forceinline__ void clear_bins(Shared& sh, int buf) {
  uint32_t* h = &sh.hist[buf][0][0];
  for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) h[i] = 0u;
  if (threadIdx.x == 0) sh.sel_bin = 0;
  __syncthreads();
}

// add one token to a bin: the 64-bit weight as two words, the carry by the value before
template <bool COUNT>
__device__ __forceinline__ void add_to_bin(Shared& sh, int buf, int bin, uint64_t W) {
  if (COUNT) atomicAdd(&sh.hist[buf][0][bin], 1u);
  const uint32_t l = static_cast<uint32_t>(W);
  const uint32_t old = atomicAdd(&sh.hist[buf][1][bin], l);
  const uint32_t h = static_cast<uint32_t>(W >> 32) + (old + l < old ? 1u : 0u);
  if (h != 0) atomicAdd(&sh.hist[buf][2][bin], h);
}

// The last bin that is not empty and before which the target is not reached (n0, e0: what lies
// before the first bin); every CTA finds the same. A bin of tokens without weight counts as
// empty where weights are asked for: no target above the weight before them is left there.
template <bool COUNT>
__device__ int find_bin(Shared& sh, int buf, int C, uint64_t target, uint64_t& n0, uint64_t& e0, uint64_t* incl, uint64_t* count) {
  const int tid = threadIdx.x;
  uint64_t n[2] = {0, 0}, w[2] = {0, 0};
  for (int c = 0; c < C; ++c) {
    const uint2 b = reinterpret_cast<const uint2*>(peer(sh.hist[buf][1], c))[tid];
    const uint2 d = reinterpret_cast<const uint2*>(peer(sh.hist[buf][2], c))[tid];
    w[0] += (static_cast<uint64_t>(d.x) << 32) + b.x;
    w[1] += (static_cast<uint64_t>(d.y) << 32) + b.y;
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
    const int j = bin & 1;
    sh.sel_e = ee[j];
    sh.sel_incl = ee[j] + w[j];
    sh.sel_n = static_cast<uint32_t>(nn[j]);
    sh.sel_cnt = static_cast<uint32_t>(n[j]);
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

// The bound of comp below which the tokens stay, COUNT: the first `target` of them, else those before
// which the weight is below `target` (> 0). Looked at: comp in [lo, lo + 2^width) with z >= z_cut,
// before which lies the weight e0. *kept gets the weight of those that stay.
template <bool COUNT, typename T>
__device__ uint64_t select(const Row<T>& row, const Scale& sc, uint64_t target, uint64_t lo, int width, uint64_t e0, float z_cut,
                           Shared& sh, int& buf, int C, uint64_t* kept) {
  uint64_t n0 = 0, count;
  for (;;) {
    const int shift = max(0, width - kBinBits);
    clear_bins(sh, buf);
    row.each([&](float x, int i) {
      const float z = fminf(x, kFltMax);
      if (!(x >= z_cut) || z == -INFINITY) return;
      const uint64_t at = comp_of(z, i, sc.kmax) - lo;       // wraps to a large number below lo
      if (at >> width != 0) return;
      float wh, wl;
      weight(z, sc, sh.tab, wh, wl);
      add_to_bin<true>(sh, buf, static_cast<int>(at >> shift), weight_int(wh, wl));
    });
    cluster_sync();
    const int bin = find_bin<COUNT>(sh, buf, C, target, n0, e0, kept, &count);
    buf ^= 1;
    lo += static_cast<uint64_t>(bin) << shift;
    if (shift == 0 || (COUNT && n0 + count <= target)) return lo + (1ull << shift);
    width = shift;
  }
}

// sort the first P (a power of two, 32 <= P <= kMerged) of sh.sort ascending
__device__ void sort_merged(Shared& sh, int P) {
  const int tid = threadIdx.x;
  for (int k = 2; k <= P; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (j < 32) {
        // the rest of this merge stays within a warp's 32 neighbours
        for (int i = tid; i < P; i += kThreads) {
          uint64_t v = sh.sort[i];
          for (int d = j; d > 0; d >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, v, d);
            const bool up = (i & k) == 0, low = (i & d) == 0;
            v = (up == low) == (o < v) ? o : v;
          }
          sh.sort[i] = v;
        }
        __syncthreads();
        break;
      }
      for (int t = tid; t < P / 2; t += kThreads) {
        const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1));
        const uint64_t a = sh.sort[i], b = sh.sort[i + j];
        if (((i & k) == 0) == (b < a)) {
          sh.sort[i] = b;
          sh.sort[i + j] = a;
        }
      }
      __syncthreads();
    }
  }
}

__device__ __forceinline__ int padded(int n) {
  int P = 32;
  while (P < n) P <<= 1;
  return P;
}

// The tokens f picks, as comp, of all CTAs in sh.sort, sorted; returns their number, or -1 where they are
// too many. Every CTA gets the same.
template <typename T, typename F>
__device__ int gather(const Row<T>& row, const Scale& sc, Shared& sh, int C, F f) {
  const int tid = threadIdx.x;
  if (tid == 0) sh.list_n = 0;
  __syncthreads();
  row.each([&](float x, int i) {
    if (!f(x, i)) return;
    const uint32_t at = atomicAdd(&sh.list_n, 1u);
    if (at < kList) sh.list[at] = comp_of(fminf(x, kFltMax), i, sc.kmax);
  });
  cluster_sync();
  uint32_t n = 0;
  bool fits = true;
  for (int c = 0; c < C; ++c) {
    const uint32_t k = *peer(&sh.list_n, c);
    fits = fits && k <= kList;
    n += k;
  }
  fits = fits && n <= kMerged;
  if (fits) {
    const int P = padded(static_cast<int>(n));
    uint32_t at = 0;
    for (int c = 0; c < C; ++c) {
      const uint32_t k = *peer(&sh.list_n, c);
      const uint64_t* from = peer(sh.list, c);
      for (uint32_t i = tid; i < k; i += kThreads) sh.sort[at + i] = from[i];
      at += k;
    }
    for (int i = static_cast<int>(n) + tid; i < P; i += kThreads) sh.sort[i] = kAll;
    __syncthreads();
    sort_merged(sh, P);
  }
  return fits ? static_cast<int>(n) : -1;
}

// Of the n sorted tokens in sh.sort, before which lies the weight e0: those that stay, in their order,
// under `k` tokens, the sum before a token below ceil(top_p * sum of the first k) (or below
// `target`, where that is > 0) and min-p. *kept: e0 and their weight. At least one stays.
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
      const float z = okey_value(sc.kmax - static_cast<uint32_t>(sh.sort[j] >> kIdxBits));
      float wh, wl;
      weight(z, sc, sh.tab, wh, wl);
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
  block_scan(static_cast<uint64_t>(stay), sh.part2, &total);
  const int m = static_cast<int>(total);
  block_scan(mine, sh.part, &total);
  *kept = e0 + total;
  return m;
}

// grid (rows * C), clusters of C CTAs: one row each
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_sample(Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  constexpr int VE = Row<T>::VE;
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
  const uint8_t* start = static_cast<const uint8_t*>(p.logits) + r * p.row_bytes;
  Row<T> row;
  row.off = static_cast<int>((reinterpret_cast<uintptr_t>(start) & 15) / sizeof(T));
  row.base = start - row.off * sizeof(T);
  row.V = p.V;
  row.nres = p.nres;
  row.data = reinterpret_cast<uint4*>(smem);
  const int nvec = (row.off + p.V + VE - 1) / VE;
  row.v0 = (rank * kWarps + wid) * p.nvw;
  row.nw = max(0, min(p.nvw, nvec - row.v0));

  // every vector of this thread is on its way at once
  for (int k = lane; k < min(row.nw, row.nres); k += 32) {
    uint4* dst = row.data + wid * row.nres + k;
    const int v = row.v0 + k;
    if (row.inside(v))
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)),
                   "l"(reinterpret_cast<const uint4*>(row.base) + v)
                   : "memory");
    else
      *dst = row.edge(v);
  }
  if (tid < kTab) sh.tab[tid] = kPowers.v[tid];
  float temp = p.temperature != nullptr ? __ldg(p.temperature + set) : 1.f;
  int64_t k = p.top_k != nullptr ? __ldg(p.top_k + set) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + set) : 1.f;
  float min_p = p.min_p != nullptr ? __ldg(p.min_p + set) : 0.f;
  if (!(temp >= 0.f)) {
    if (tid == 0) record_error(p.hdr, SSD_ERR_DEVICE, 501);
    temp = 0.f;
  }
  temp = fminf(temp, 0x1p100f);
  if (temp == 0.f) {                       // greedy: the first of the largest
    temp = 1.f;
    k = 1;
  }
  min_p = fminf(min_p, 1.f);
  if (k < 0 || k >= p.V) k = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");

  // ---- the row's largest value; with top-k also a value that k tokens at least reach: the smallest,
  // over the CTAs, of the ceil(k / C)-th largest of the threads' own maxima
  float mx = -INFINITY;
  row.each([&](float x, int) { mx = fmaxf(mx, x); });
  mx = fminf(mx, kFltMax);
  {
    const float m = warp_max(mx);
    if (lane == 0) sh.wmax[wid] = m;
  }
  __syncthreads();
  uint32_t reach = 0;
  const int64_t share = (k + C - 1) / C;
  if (k > 0 && share <= kThreads) {
    const uint32_t key = okey(mx + 0.f);
    for (int bit = 31; bit >= 10; --bit) {
      const uint32_t t = reach | (1u << bit);
      if (__syncthreads_count(key >= t) >= share) reach = t;
    }
  }
  if (tid < C) {
    float t = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t = fmaxf(t, sh.wmax[w]);
    *peer(&sh.ex_max[rank], tid) = t;
    *peer(&sh.ex_key[rank], tid) = reach;
  }
  cluster_sync();
  float zmax = -INFINITY;
  for (int c = 0; c < C; ++c) {
    zmax = fmaxf(zmax, sh.ex_max[c]);
    reach = min(reach, sh.ex_key[c]);
  }
  const bool empty = !(zmax > -INFINITY);
  const Scale sc = make_scale(zmax, temp);

  uint64_t bound = kAll, S = 0, before = 0, mine = 0;
  bool known = false, all_cut = false;       // S is that of the tokens that stay; min-p is in the bound
  if (!empty) {
    int buf = 0;
    if (k > 0) {
      const float low = reach > okey(-INFINITY) ? okey_value(reach) : -INFINITY;
      const int n = gather(row, sc, sh, C, [&](float x, int) { return x >= low && x > -INFINITY; });
      if (n >= 0) {
        const int m = cut_sorted(sh, sc, n, 0, static_cast<int>(k), top_p, 0, min_p, &S);
        bound = sh.sort[m - 1] + 1;
        all_cut = true;
      } else {
        bound = select<true>(row, sc, static_cast<uint64_t>(k), 0, 32 + kIdxBits, 0, low, sh, buf, C, &S);
      }
      known = true;
    }
    if (top_p < 1.f && !all_cut) {
      // tokens of a weight below (1 - top_p) / V, together, are not more than the tail that is cut
      // (the sum is at least 1); binned are the others, and all are summed
      const float low = __fadd_rd(zmax, __fmul_rd(logf((1.f - fmaxf(top_p, 0.f)) / static_cast<float>(p.V) * 0.999f), temp));
      const float z_cut = fmaxf(low, sc.zmin);
      const uint32_t kd_cut = sc.kmax - okey(z_cut + 0.f);
      const int width = 32 - __clz(kd_cut | 1) + kIdxBits;
      const int shift = width - kBinBits;
      clear_bins(sh, buf);
      int sa = 0, sb = 0;
      row.each([&](float x, int i) {
        float wh, wl;
        int a, b;
        weight(x, sc, sh.tab, wh, wl);
        weight_parts(wh, wl, a, b);
        sa += a - kMagicBits;
        sb += b - kMagicBits;
        if (x >= z_cut)
          add_to_bin<false>(sh, buf, static_cast<int>(comp_of(fminf(x, kFltMax), i, sc.kmax) >> shift),
                            static_cast<uint64_t>(static_cast<int64_t>(a - kMagicBits) * 4194304 + (b - kMagicBits)));
      });
      const uint64_t sum = cluster_sum(static_cast<uint64_t>(static_cast<int64_t>(sa) * 4194304 + sb), sh, 0, rank, C, &before, &mine);
      const uint64_t target = max(mul_fraction(known ? S : sum, fmaxf(top_p, 0.f), true), uint64_t{1});
      uint64_t n0 = 0, e0 = 0, incl, count;
      const uint64_t lo = static_cast<uint64_t>(find_bin<false>(sh, buf, C, target, n0, e0, &incl, &count)) << shift;
      buf ^= 1;
      const int n = gather(row, sc, sh, C, [&](float x, int i) {
        return x >= z_cut && (comp_of(fminf(x, kFltMax), i, sc.kmax) - lo) >> shift == 0;
      });
      if (n >= 0) {
        const int m = cut_sorted(sh, sc, n, e0, n, 1.f, target, 0.f, &S);
        bound = sh.sort[m - 1] + 1;
      } else {
        bound = select<false>(row, sc, target, lo, shift, e0, z_cut, sh, buf, C, &S);
      }
      known = true;
    }
  }
  // kept: z > zt, or z == zt and index < it
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
  const bool use_min_p = min_p > 0.f && !all_cut;
  // the weight of a token that stays; false for the others (NaN among them)
  auto kept_weight = [&](float x, int i, float& wh, float& wl) {
    wh = wl = 0.f;
    const float z = fminf(x, kFltMax);
    if (!(z > zt || (z == zt && i < it)) || !(x >= sc.zmin)) return false;
    weight(x, sc, sh.tab, wh, wl);
    if (use_min_p && !(x >= sc.zmax || (wh - min_p) + wl >= 0.f)) {
      wh = wl = 0.f;
      return false;
    }
    return true;
  };

  const bool draw = p.token != nullptr && !empty;
  if (!empty && (use_min_p || !known || draw)) {
    uint64_t t = 0;
    row.each([&](float x, int i) {
      float wh, wl;
      if (kept_weight(x, i, wh, wl)) t += weight_int(wh, wl);
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
  auto probability = [&](float wh, float wl) { return fmaf(wh, ih, fmaf(wh, il, wl * ih)); };

  if (p.probs != nullptr) {
    float* out = p.probs + r * p.V;
    const bool wide = ((reinterpret_cast<uintptr_t>(out) / 4 - row.off) & 3) == 0;
    if (wide) {
      for (int kv = lane; kv < row.nw; kv += 32) {
        const uint4 q = row.get(wid, row.v0, kv);
        const int i = (row.v0 + kv) * VE - row.off;
        float v[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          float wh, wl;
          kept_weight(Row<T>::elem(q, e), i + e, wh, wl);
          v[e] = probability(wh, wl);
        }
        if (row.inside(row.v0 + kv) && in_range(i + VE - 1, p.V, p.hdr, 510)) {
#pragma unroll
          for (int e = 0; e < VE; e += 4) *reinterpret_cast<float4*>(out + i + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (i + e >= 0 && i + e < p.V) out[i + e] = v[e];
        }
      }
    } else {
      // rows whose elements lie otherwise in 16 bytes than the output's: four bytes a lane
      const int i0 = row.v0 * VE - row.off;
      for (int j = lane; j < row.nw * VE; j += 32) {
        const int i = i0 + j;
        if (i < 0 || i >= p.V || !in_range(i, p.V, p.hdr, 511)) continue;
        const int kv = j / VE;
        const T* src = kv < row.nres ? reinterpret_cast<const T*>(row.data + wid * row.nres) + j
                                     : reinterpret_cast<const T*>(row.base) + static_cast<int64_t>(row.v0) * VE + j;
        float x, wh, wl;
        if constexpr (sizeof(T) == 4) x = *src; else x = bf16_to_f32(*src);
        kept_weight(x, i, wh, wl);
        out[i] = probability(wh, wl);
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
    if (thr >= before && thr < before + mine) {
      // this CTA holds it: the warp, then the vector, then the element
      uint64_t c0 = before;
      int w = 0;
      while (w < kWarps - 1 && thr >= c0 + sh.wsum[w]) c0 += sh.wsum[w++];
      const int first = (rank * kWarps + w) * p.nvw;
      const int nw = max(0, min(p.nvw, nvec - first));
      for (int k0 = 0; k0 < nw; k0 += kThreads) {
        const int kk = k0 + tid;
        uint4 q = make_uint4(0, 0, 0, 0);
        uint64_t t = 0, all;
        const int i = (first + kk) * VE - row.off;
        if (kk < nw) {
          q = row.get(w, first, kk);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            float wh, wl;
            if (kept_weight(Row<T>::elem(q, e), i + e, wh, wl)) t += weight_int(wh, wl);
          }
        }
        uint64_t pre = c0 + block_scan(t, sh.part, &all);
        if (thr >= pre && thr < pre + t) {
          bool done = false;
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            float wh, wl;
            if (!done && kept_weight(Row<T>::elem(q, e), i + e, wh, wl)) {
              pre += weight_int(wh, wl);
              if (thr < pre) {
                done = true;
                p.token[r] = i + e;
                if (p.prob != nullptr) p.prob[r] = probability(wh, wl);
              }
            }
          }
        }
        c0 += all;
        if (thr < c0) break;
      }
    }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

template <typename T>
static int launch(const Params& in, int64_t rows, cudaStream_t s) {
  constexpr int VE = Row<T>::VE;
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  static int sms[kMaxDevices];
  constexpr int kMaxData = 160 * 1024;
  const int dev = current_device();
  if (dev < 0) return SSD_ERR_CUDA;
  std::call_once(once[dev], [dev] {
    err[dev] = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxData);
    if (err[dev] == cudaSuccess) err[dev] = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
  });
  if (err[dev] != cudaSuccess) return SSD_ERR_CUDA;
  Params p = in;
  const int nvec = (p.V + 2 * VE - 2) / VE;                  // at most, whatever the row's first element's place
  int C = 1;
  while (C < kMaxCluster && (16LL * nvec / C > 72 * 1024 || (rows * C * 2 <= 2LL * sms[dev] && nvec / C > 4 * kThreads))) C *= 2;
  const int per = kWarps * C;
  p.nvw = (nvec + per - 1) / per;
  p.nvw = (p.nvw + 31) / 32 * 32;
  p.nres = std::min(p.nvw, kMaxData / 16 / kWarps);
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
    if (cudaLaunchKernelEx(&cfg, k_sample<T>, p) != cudaSuccess) return SSD_ERR_CUDA;
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
