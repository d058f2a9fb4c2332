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
  float2 tab[kTab];                        // 2^(i/64) as high and low fp32
  uint32_t hist[2][3][kBins];              // count, low and high word of the weight; two levels in turns
  uint64_t ex_sum[2][kMaxCluster];         // from every CTA of the cluster
  float ex_max[kMaxCluster];
  uint64_t part[kWarps], part2[kWarps];
  uint64_t wsum[kWarps];
  float wmax[kWarps];
  uint64_t sel_e, sel_incl;                // of the bin chosen: weight before it, and with it
  uint32_t sel_n, sel_cnt, sel_bin, any;
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

// NaN counts as -inf, +inf as the largest finite number, -0 as 0
__device__ __forceinline__ float norm(float z) { return z > -INFINITY ? fminf(z, 3.402823466e38f) + 0.f : -INFINITY; }

struct Scale {
  float zmax, ch, cl;                      // ch + cl = log2(e) / T
};

// w = wh + wl, relative error under 2^-29; 0 below 2^-125
__device__ __forceinline__ bool weight(float z, const Scale& s, const float2* tab, float& wh, float& wl) {
  const float dh = z - s.zmax;
  const float ph = dh * s.ch;
  wh = wl = 0.f;
  if (!(ph >= -125.f)) return false;
  const float bb = dh - z;
  const float dl = (z - (dh - bb)) + (-s.zmax - bb);         // z - zmax = dh + dl exactly
  const float pl = fmaf(dl, s.ch, fmaf(dh, s.cl, fmaf(dh, s.ch, -ph)));
  const float m = fmaf(ph, static_cast<float>(kTab), 12582912.f);
  const int n = __float_as_int(m) - 0x4B400000;              // ph = n / 64 + r
  const float r = fmaf(m - 12582912.f, -1.f / kTab, ph) + pl;
  // 2^r - 1 for |r| <= 1/128: the powers of ln 2 over factorials, the next term is below 4e-11
  const float q = fmaf(fmaf(0.0555041087f, r, 0.2402265070f), r, 0.6931471806f);
  const float2 t = tab[n & (kTab - 1)];
  const float s2 = __uint_as_float(static_cast<uint32_t>(127 + (n >> 6)) << 23);
  wh = t.x * s2;
  // ln 2 to fp32 is off by 1.9e-9 relative: its rest times r
  wl = fmaf(wh, fmaf(q, r, -1.9046542e-9f * r), t.y * s2);
  return true;
}

// round(w 2^43) for w <= 1
__device__ __forceinline__ uint64_t weight_int(float wh, float wl) {
  const float a = fmaf(wh + wl, 2097152.f, 12582912.f);
  const float lo = fmaf(a - 12582912.f, -1.f / 2097152.f, wh) + wl;
  const float b = fmaf(lo, 8796093022208.f, 12582912.f);
  return static_cast<uint64_t>(static_cast<int64_t>(__float_as_int(a) - 0x4B400000) * 4194304 +
                               (__float_as_int(b) - 0x4B400000));
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
  // f(value, index) for every element of this warp
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int k = lane; k < nw; k += 32) {
      const uint4 q = get(w, v0, k);
      const int i = (v0 + k) * VE - off;
#pragma unroll
      for (int e = 0; e < VE; ++e) f(norm(elem(q, e)), i + e);
    }
  }
};

// sum over the cluster of one number a thread; *mine gets this CTA's. Slot `ex` is written once.
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

// The bound of comp below which the tokens stay: with `by_count` the first `target` of them, else
// those before which the weight is below `target` (> 0). Only comp < range is looked at.
// *kept gets the weight of those that stay. Every CTA of the cluster finds the same.
template <typename T>
__device__ uint64_t select(const Row<T>& row, const Scale& sc, uint32_t kmax, bool by_count, uint64_t target, int range_bits,
                           float z_cut, Shared& sh, int& buf, int C, uint64_t* kept) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  uint64_t lo = 0, e0 = 0;
  uint64_t n0 = 0;
  int width = range_bits;                                    // the bins cover comp in [lo, lo + 2^width)
  for (;;) {
    const int shift = max(0, width - kBinBits);
    uint32_t* cnt = sh.hist[buf][0];
    uint32_t* wlo = sh.hist[buf][1];
    uint32_t* whi = sh.hist[buf][2];
    for (int i = tid; i < kBins; i += kThreads) cnt[i] = wlo[i] = whi[i] = 0u;
    if (tid == 0) sh.sel_bin = 0;
    __syncthreads();
    row.each([&](float z, int i) {
      if (z < z_cut || z == -INFINITY) return;
      const uint64_t comp = (static_cast<uint64_t>(kmax - okey(z)) << kIdxBits) + static_cast<uint32_t>(i);
      if (comp < lo || (comp - lo) >> width != 0) return;
      const int bin = static_cast<int>((comp - lo) >> shift);
      float wh, wl;
      weight(z, sc, sh.tab, wh, wl);
      const uint64_t W = weight_int(wh, wl);
      atomicAdd(&cnt[bin], 1u);
      const uint32_t l = static_cast<uint32_t>(W);
      const uint32_t old = atomicAdd(&wlo[bin], l);
      const uint32_t h = static_cast<uint32_t>(W >> 32) + (old + l < old ? 1u : 0u);
      if (h != 0) atomicAdd(&whi[bin], h);
    });
    cluster_sync();
    // two bins a thread, summed over the cluster, then a scan over the threads
    uint64_t n[2] = {0, 0}, w[2] = {0, 0};
    for (int c = 0; c < C; ++c) {
      const uint2 a = reinterpret_cast<const uint2*>(peer(cnt, c))[tid];
      const uint2 b = reinterpret_cast<const uint2*>(peer(wlo, c))[tid];
      const uint2 d = reinterpret_cast<const uint2*>(peer(whi, c))[tid];
      n[0] += a.x;
      n[1] += a.y;
      w[0] += (static_cast<uint64_t>(d.x) << 32) + b.x;
      w[1] += (static_cast<uint64_t>(d.y) << 32) + b.y;
    }
    const uint64_t nt = n[0] + n[1], wt = w[0] + w[1];
    uint64_t ns = nt, wsm = wt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, ns, o), y = __shfl_up_sync(0xffffffffu, wsm, o);
      if (lane >= o) {
        ns += x;
        wsm += y;
      }
    }
    if (lane == 31) {
      sh.part[wid] = ns;
      sh.part2[wid] = wsm;
    }
    __syncthreads();
    uint64_t nb = n0, eb = e0;
    for (int i = 0; i < wid; ++i) {
      nb += sh.part[i];
      eb += sh.part2[i];
    }
    nb += ns - nt;
    eb += wsm - wt;
    // the last bin that holds a token and before which the target is not reached
    uint64_t nn[2] = {nb, nb + n[0]}, ee[2] = {eb, eb + w[0]};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (n[j] > 0 && (by_count ? nn[j] : ee[j]) < target) atomicMax(&sh.sel_bin, static_cast<uint32_t>(2 * tid + j));
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
    const uint64_t incl = sh.sel_incl;
    const uint32_t count = sh.sel_cnt;
    n0 = sh.sel_n;
    e0 = sh.sel_e;
    buf ^= 1;
    lo += static_cast<uint64_t>(bin) << shift;
    if (shift == 0 || count <= 1 || (by_count && n0 + count <= target)) {
      *kept = incl;
      return lo + (1ull << shift);
    }
    width = shift;
  }
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
  if (tid < kTab) {
    const double x = exp2(static_cast<double>(tid) / kTab);
    sh.tab[tid].x = static_cast<float>(x);
    sh.tab[tid].y = static_cast<float>(x - sh.tab[tid].x);
  }
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
  min_p = fminf(min_p, 1.f);
  if (k < 0 || k >= p.V) k = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");

  // ---- the row's largest value
  float mx = -INFINITY;
  row.each([&](float z, int) { mx = fmaxf(mx, z); });
  mx = warp_max(mx);
  if (lane == 0) sh.wmax[wid] = mx;
  __syncthreads();
  if (tid < C) {
    float t = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t = fmaxf(t, sh.wmax[w]);
    *peer(&sh.ex_max[rank], tid) = t;
  }
  cluster_sync();
  Scale sc;
  sc.zmax = -INFINITY;
  for (int c = 0; c < C; ++c) sc.zmax = fmaxf(sc.zmax, sh.ex_max[c]);
  const bool empty = !(sc.zmax > -INFINITY);
  const double c2 = fmin(1.4426950408889634 / static_cast<double>(temp), 0x1p120);
  sc.ch = static_cast<float>(c2);
  sc.cl = static_cast<float>(c2 - sc.ch);
  const uint32_t kmax = okey(sc.zmax);

  uint64_t bound = kAll, S = 0, before = 0, mine = 0;
  bool known = false;
  if (!empty) {
    int buf = 0;
    if (k > 0) {
      bound = select(row, sc, kmax, true, static_cast<uint64_t>(k), 32 + kIdxBits, -INFINITY, sh, buf, C, &S);
      known = true;
    }
    if (top_p < 1.f && k != 1) {
      if (!known) {
        uint64_t t = 0;
        row.each([&](float z, int) {
          float wh, wl;
          if (weight(z, sc, sh.tab, wh, wl)) t += weight_int(wh, wl);
        });
        S = cluster_sum(t, sh, 0, rank, C, &before, &mine);
      }
      uint64_t target = mul_fraction(S, fmaxf(top_p, 0.f), true);
      if (target < 1) target = 1;
      bound = select(row, sc, kmax, false, target, 32 + kIdxBits, -INFINITY, sh, buf, C, &S);
      known = true;
    }
  }
  // kept: z > zt, or z == zt and index < it
  float zt = -INFINITY;
  int it = 0;
  if (bound != kAll) {
    const uint64_t kd = bound >> kIdxBits;
    if (kd < kmax - okey(-INFINITY)) {
      const uint32_t key = kmax - static_cast<uint32_t>(kd);
      it = static_cast<int>(bound & ((1u << kIdxBits) - 1));
      // the key of -0, which no element has, as a bound means all zeros
      if (key == 0x7fffffffu) it = p.V;
      zt = okey_value(key) + 0.f;
    }
  }
  auto keep = [&](float z, int i) { return z > zt || (z == zt && i < it && z > -INFINITY); };
  // its weight, where it also passes min-p
  auto kept_weight = [&](float z, int i, float& wh, float& wl) {
    wh = wl = 0.f;
    if (!keep(z, i) || !weight(z, sc, sh.tab, wh, wl)) return false;
    if (min_p > 0.f && !((wh - min_p) + wl >= 0.f)) {
      wh = wl = 0.f;
      return false;
    }
    return true;
  };

  if (!empty && (min_p > 0.f || !known || p.token != nullptr)) {
    uint64_t t = 0;
    row.each([&](float z, int i) {
      float wh, wl;
      if (kept_weight(z, i, wh, wl)) t += weight_int(wh, wl);
    });
    S = cluster_sum(t, sh, 1, rank, C, &before, &mine);
  }
  const double inv = S > 0 ? 8796093022208.0 / static_cast<double>(S) : 0.0;
  const float ih = static_cast<float>(inv), il = static_cast<float>(inv - ih);
  auto probability = [&](float wh, float wl) { return fmaf(wh, ih, fmaf(wh, il, wl * ih)); };

  if (p.probs != nullptr) {
    float* out = p.probs + r * p.V;
    // this warp's elements side by side, four bytes a lane
    const int i0 = row.v0 * VE - row.off;
    for (int j = lane; j < row.nw * VE; j += 32) {
      const int i = i0 + j;
      if (i < 0 || i >= p.V || !in_range(i, p.V, p.hdr, 510)) continue;
      const int kv = j / VE;
      const T* src = kv < row.nres ? reinterpret_cast<const T*>(row.data + wid * row.nres) + j
                                   : reinterpret_cast<const T*>(row.base) + static_cast<int64_t>(row.v0) * VE + j;
      float z;
      if constexpr (sizeof(T) == 4) z = norm(*src); else z = norm(bf16_to_f32(*src));
      float wh, wl;
      kept_weight(z, i, wh, wl);
      out[i] = probability(wh, wl);
    }
  }

  if (p.token != nullptr) {
    if (empty) {
      if (rank == 0 && tid == 0) {
        p.token[r] = -1;
        if (p.prob != nullptr) p.prob[r] = 0.f;
      }
    } else {
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
          uint64_t t = 0;
          const int i = (first + kk) * VE - row.off;
          if (kk < nw) {
            q = row.get(w, first, kk);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              float wh, wl;
              if (kept_weight(norm(Row<T>::elem(q, e)), i + e, wh, wl)) t += weight_int(wh, wl);
            }
          }
          uint64_t x = t;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          __syncthreads();
          if (lane == 31) sh.part[wid] = x;
          __syncthreads();
          uint64_t pre = c0, all = c0;
          for (int j = 0; j < kWarps; ++j) {
            if (j < wid) pre += sh.part[j];
            all += sh.part[j];
          }
          pre += x - t;
          if (thr >= pre && thr < pre + t) {
            bool done = false;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              float wh, wl;
              if (!done && kept_weight(norm(Row<T>::elem(q, e)), i + e, wh, wl)) {
                pre += weight_int(wh, wl);
                if (thr < pre) {
                  done = true;
                  p.token[r] = i + e;
                  if (p.prob != nullptr) p.prob[r] = probability(wh, wl);
                }
              }
            }
          }
          c0 = all;
          if (thr < c0) break;
        }
      }
    }
  }
  // no CTA leaves while another may still read its histograms
  cluster_sync();
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
