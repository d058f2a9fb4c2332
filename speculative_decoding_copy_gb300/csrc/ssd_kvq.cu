// Writers of the 8-bit key/value cache: rows quantised into e4m3 codes with a power-of-two
// scale for each block of tokens and head.
//
// A power of two costs an e4m3 number nothing (its precision is relative) and makes a
// grown scale exact on the codes already there: only those that fall below the smallest
// normal code round a second time.
//
// A group of warps, one for each 16 tokens of a scale block, quantises one run (the rows that go to
// one block) of one head, of the keys or of the values: the rows are read once into registers
// (up to eight 16-byte words a thread cover the block's rows x 128 elements), their largest
// magnitude is reduced over the group, and the codes leave as 8 bytes a word, contiguous over
// the run.
//
// What bounds them: the bytes of the rows, and for a few tokens the launch. 21 384 prompt rows
// of 8 kv heads (131 MB) take 24 us where L2 still holds part of them, as behind a projection, and
// 31.3 from cold caches, 4.2 TB/s of the 6.8 that a plain copy reaches: a CTA reads
// its 32 KB, waits for the maximum of all of it, and writes; five CTAs an SM, a few registers of
// theirs spilled, fill each other's waits better than four without (31.3 us from cold caches, 34.5),
// six worse; with smaller blocks, whose groups are not tied to each other, four do (33.9, five 42).
// Blocks of 16 tokens take 33.9 us by a warp each, where one run after another by all of a CTA took
// 101, fp32 rows 54 and 205. Replayed from a graph 64 single tokens take 5.4 us, the accepted tokens of
// one sequence and of 32 sequences 2.5: little more than an empty kernel.
#include <type_traits>

#include "ssd_kvq.cuh"

namespace ssd {

constexpr int kQuantThreads = 256;
constexpr int kMaxScaleBlock = 128;
constexpr int kGroupRows = 16;          // rows of a run that a warp takes

struct QuantDst {
  uint8_t* codes;       // place 0 of the block, [scale_block][dh]
  float* scale;
  int row;              // first place written
};

// the least power of two s with a <= 448 s (448 = 1.75 * 2^8), at least 2^-100; a as bits
__device__ __forceinline__ float pow2_scale(uint32_t a) {
  const int e = static_cast<int>(a >> 23) - 127;
  const int k = max((a & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7, -100);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// 1 / s where s is a power of two whose reciprocal is normal, else 0
__device__ __forceinline__ float exact_reciprocal(float s) {
  const uint32_t u = __float_as_uint(s);
  const uint32_t e = u >> 23;
  return (u & 0x7fffffu) == 0 && e >= 1 && e <= 253 ? __uint_as_float((254 - e) << 23) : 0.f;
}

// off the common path: its code is kept out of the loops
__device__ __noinline__ float divide(float x, float s) { return __fdiv_rn(x, s); }

// 8 elements of a row. top: an upper bound of their magnitudes, as fp32 bits, that is exact unless
// one is not finite (then >= 0x7f800000); finite_top: the largest finite one.
template <typename T>
struct Word;
template <>
struct Word<uint16_t> {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = max_u16x2(max_u16x2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu), max_u16x2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
};
template <>
struct Word<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    float x[8];
    get(x);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    return m;
  }
};

template <typename T>
__device__ __forceinline__ uint32_t finite_top(const Word<T>& w) {
  float x[8];
  w.get(x);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
    m = max(m, u < 0x7f800000u ? u : 0u);
  }
  return m;
}

// the W warps that work on one run
template <int W>
struct Group {
  static constexpr int kThreads = 32 * W;
  int tid;                                // this thread's number among them
  int barrier;                            // of their own
  uint32_t* red;                          // one word a warp
  __device__ __forceinline__ void sync() const {
    __syncwarp();
    if (W > 1) asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(barrier), "n"(kThreads) : "memory");
  }
};

// Quantise n rows (at most 16 a warp of the group) of dh elements, `stride` elements apart at src, into
// places d.row .. d.row + n - 1 of one block. Every thread of the group calls it.
template <typename T, int W>
__device__ __forceinline__ void quant_run(const T* __restrict__ src, int64_t stride, int n, int dh, QuantDst d,
                                          const Group<W>& grp) {
  const int tid = grp.tid, lane = tid & 31, wid = tid >> 5;
  const int sh = dh == 128 ? 4 : 3;           // 8-element words per row
  constexpr int kWords = kGroupRows * 16 / 32;
  // word i of a thread: row row0 + i * rows_step, the same place in each
  const int row0 = tid >> sh, rows_step = grp.kThreads >> sh;
  const T* p = src + row0 * stride + ((tid & ((1 << sh) - 1)) << 3);
  const int64_t step = rows_step * stride;
  const int mine = row0 < n ? min(kWords, (n - 1 - row0) / rows_step + 1) : 0;
  const float old = d.row == 0 ? 0.f : *d.scale;
  Word<T> w[kWords];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if (i < mine) w[i].load(p);
    p += step;
  }
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    if (i < mine) m = max(m, w[i].top());
  if (m >= 0x7f800000u) {
    m = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      if (i < mine) m = max(m, finite_top<T>(w[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  grp.sync();                                 // `red` and the block's scale of an earlier run
  if (lane == 0) grp.red[wid] = m;
  grp.sync();
#pragma unroll
  for (int i = 0; i < W; ++i) m = max(m, grp.red[i]);
  const float need = pow2_scale(m);
  const float now = d.row == 0 ? need : fmaxf(old, need);
  if (d.row > 0 && now > old) {
    // the rows before the run, under the grown scale
    const float ratio = __fdiv_rn(old, now);
    const int held = d.row << sh;
    for (int c = tid; c < held; c += grp.kThreads) {
      uint2* p = reinterpret_cast<uint2*>(d.codes) + c;
      const uint2 v = *p;
      const uint32_t h[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        e4m3x2_to_f32(h[i], lo, hi);
        q[i] = e4m3x2(lo * ratio, hi * ratio);
      }
      *p = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    }
  }
  uint2* out = reinterpret_cast<uint2*>(d.codes) + (d.row << sh) + tid;
  const float inv = exact_reciprocal(now);
  if (inv != 0.f) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if (i < mine) {
        float x[8];
        w[i].get(x);
        out[i * grp.kThreads] = make_uint2(e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                            e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
      }
    }
  } else {
    // a scale that is no power of two: the caller's own, which this run left as it was
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if (i < mine) {
        float x[8];
        w[i].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = divide(x[e], now);
        out[i * grp.kThreads] = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
      }
    }
  }
  grp.sync();                                 // every thread has read the old scale
  if (tid == 0) *d.scale = now;
}

// grid (row ranges of `range` rows) x (heads, keys / values), the latter fastest, so that the CTAs
// that share rows (and DRAM pages of a projection's output) run together: the runs that start
// in the range, dealt to the groups in turn
template <typename T, int W>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? (W == 8 ? 5 : 4) : 2)
k_append_quant(ssd_append_quant_args a, int range, WsHeader* hdr) {
  constexpr int sb_log2 = W == 1 ? 4 : W == 2 ? 5 : W == 4 ? 6 : 7;     // 16 tokens a warp
  __shared__ int32_t slot[2 * kMaxScaleBlock];
  constexpr int kMasks = 2 * kMaxScaleBlock / 32;
  __shared__ uint32_t brk[kMasks];                      // rows that do not continue the row before
  __shared__ uint32_t start[kMasks];                    // ... and have a slot
  __shared__ uint32_t red[kQuantThreads / 32];
  constexpr int kGroups = kQuantThreads / Group<W>::kThreads;
  const int mine = static_cast<int>(threadIdx.x) / Group<W>::kThreads;
  const Group<W> grp = {static_cast<int>(threadIdx.x) % Group<W>::kThreads, 1 + mine, red + mine * W};
  static_assert(kQuantThreads == 2 * kMaxScaleBlock, "one thread a row of the window");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(2 * a.Hkv));
  const bool is_v = part >= a.Hkv;
  const int h = is_v ? part - a.Hkv : part;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(2 * a.Hkv)) * range;
  constexpr int sb = 1 << sb_log2;
  const int window = range + sb;                        // a run that starts in the range ends here
  // one thread a row: its slot, and whether it continues the run of the row before
  const int64_t t = t0 + tid;
  const int64_t pool = a.num_pages * a.page_tokens;
  int32_t s = -1, before = -2;
  if (tid < window && t < a.T) {
    s = a.slot_map[t];
    if (t > 0) before = a.slot_map[t - 1];
    if (s >= pool) {
      if (h == 0 && !is_v && tid < range) record_error(hdr, SSD_ERR_DEVICE, 420);
      s = -1;
    }
  }
  const uint32_t page_tokens = static_cast<uint32_t>(a.page_tokens);      // under 2^31, as every slot
  const uint32_t place = s >= 0 ? static_cast<uint32_t>(s) % page_tokens : 0;
  const bool cont = s >= 0 && before == s - 1 && (place & (sb - 1)) != 0;
  slot[tid] = s;
  const uint32_t word = __ballot_sync(0xffffffffu, !cont);
  const uint32_t begins = __ballot_sync(0xffffffffu, !cont && s >= 0 && tid < range);
  if ((tid & 31) == 0) {
    brk[tid >> 5] = word;
    start[tid >> 5] = begins;
  }
  __syncthreads();
  const T* src = static_cast<const T*>(is_v ? a.v_new : a.k_new) + static_cast<int64_t>(h) * a.dh;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int64_t blocks = (a.page_tokens + sb - 1) >> sb_log2;
  int run = 0;
  for (int q = 0; q < kMasks; ++q) {
    for (uint32_t left = start[q]; left != 0; left &= left - 1) {
      if (run++ % kGroups != mine) continue;
      const int first = q * 32 + __ffs(static_cast<int>(left)) - 1;
      // the next break ends the run (rows outside the list or the window are breaks)
      int wd = q;
      uint32_t bits = brk[wd] & ~(0xffffffffu >> (31 - (first & 31)));
      while (bits == 0 && wd + 1 < kMasks) bits = brk[++wd];
      const int last = bits != 0 ? wd * 32 + __ffs(static_cast<int>(bits)) - 1 : 2 * kMaxScaleBlock;
      const int32_t s0 = slot[first];
      const uint32_t page = static_cast<uint32_t>(s0) / page_tokens;
      const int off = static_cast<int>(static_cast<uint32_t>(s0) - page * page_tokens);
      const int blk = off >> sb_log2;
      const int64_t ph = static_cast<int64_t>(page) * a.Hkv + h;
      QuantDst d;
      d.codes = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                (ph * a.page_tokens + (static_cast<int64_t>(blk) << sb_log2)) * a.dh;
      d.scale = (is_v ? a.v_scale : a.k_scale) + ph * blocks + blk;
      d.row = off & (sb - 1);
      if (!in_range(page, a.num_pages, hdr, 421) || !in_range(off + last - first - 1, a.page_tokens, hdr, 422) ||
          !in_range(d.row + last - first - 1, sb, hdr, 423) || !in_range(t0 + last - 1, a.T, hdr, 424))
        continue;
      quant_run<T, W>(src + (t0 + first) * stride, stride, last - first, a.dh, d, grp);
    }
  }
}

// grid (sequences, heads, (keys / values) x blocks a run of Dmax rows can touch)
template <typename T, int W>
__global__ void __launch_bounds__(32 * W)
k_commit_quant(ssd_commit_quant_args a, int64_t page_tokens, int segs, WsHeader* hdr) {
  constexpr int sb_log2 = W == 1 ? 4 : W == 2 ? 5 : W == 4 ? 6 : 7;     // 16 tokens a warp
  __shared__ uint32_t red[W];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const Group<W> grp = {tid, 0, red};
  const int b = blockIdx.x, h = blockIdx.y;
  const bool is_v = static_cast<int>(blockIdx.z) >= segs;
  const int seg = static_cast<int>(blockIdx.z) - (is_v ? segs : 0);
  const bool teller = h == 0 && blockIdx.z == 0 && tid == 0;
  const int k = a.best_blk[b];
  const int64_t n = k >= 0 ? static_cast<int64_t>(a.n_out[b]) - 1 : 0;
  const int64_t P = a.prefix_len[b];
  const int64_t room = a.block_table != nullptr ? static_cast<int64_t>(a.pages_per_seq) * kPageTokens : a.P_max;
  bool ok = k < a.NB && n <= a.Dmax && P >= 0 && (n <= 0 || P + n <= room);
  if (ok && n > 0 && a.block_table != nullptr) {
    for (int64_t j = P / kPageTokens; j <= (P + n - 1) / kPageTokens; ++j) {
      const int32_t pg = a.block_table[static_cast<int64_t>(b) * a.pages_per_seq + j];
      ok = ok && pg >= 0 && pg < a.num_pages;
    }
  }
  if (teller) {
    if (!ok) record_error(hdr, SSD_ERR_DEVICE, 430);
    a.new_len[b] = static_cast<int32_t>(ok && n > 0 ? P + n : P);
  }
  if (!ok || n <= 0) return;
  // the seg-th block that the run touches: positions [p0, p1)
  const int64_t blk = (P >> sb_log2) + seg;
  const int64_t p0 = max(P, blk << sb_log2), p1 = min(P + n, (blk + 1) << sb_log2);
  if (p0 >= p1) return;
  int64_t page = b, place = p0;
  if (a.block_table != nullptr) {
    page = a.block_table[static_cast<int64_t>(b) * a.pages_per_seq + p0 / kPageTokens];
    place = p0 % kPageTokens;
  }
  const int64_t ph = page * a.Hkv + h;
  const int64_t blocks = (page_tokens + (1 << sb_log2) - 1) >> sb_log2;
  const int64_t pblk = place >> sb_log2;
  QuantDst d;
  d.codes = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (ph * page_tokens + (pblk << sb_log2)) * a.dh;
  d.scale = (is_v ? a.v_scale : a.k_scale) + ph * blocks + pblk;
  d.row = static_cast<int>(place) & ((1 << sb_log2) - 1);
  const int64_t src_row = static_cast<int64_t>(b) * a.NB * a.Dmax + static_cast<int64_t>(k) * a.Dmax + (p0 - P);
  const int64_t stride = static_cast<int64_t>(a.Hkv) * a.dh;
  if (!in_range(page, a.block_table != nullptr ? a.num_pages : a.B, hdr, 431) ||
      !in_range(place + p1 - p0 - 1, page_tokens, hdr, 432) || !in_range(d.row + p1 - p0 - 1, 1 << sb_log2, hdr, 433) ||
      !in_range(src_row + p1 - p0 - 1, static_cast<int64_t>(a.B) * a.NB * a.Dmax, hdr, 434))
    return;
  quant_run<T, W>(static_cast<const T*>(is_v ? a.v_cand : a.k_cand) + src_row * stride + static_cast<int64_t>(h) * a.dh,
               stride, static_cast<int>(p1 - p0), a.dh, d, grp);
}

// `launch` with the warps of a group as a constant
template <typename F>
static cudaError_t by_warps(int scale_block, F launch) {
  switch (scale_block) {
    case 16: return launch(std::integral_constant<int, 1>());
    case 32: return launch(std::integral_constant<int, 2>());
    case 64: return launch(std::integral_constant<int, 4>());
    default: return launch(std::integral_constant<int, 8>());
  }
}

}  // namespace ssd

extern "C" int ssd_append_kv_quant(const ssd_append_quant_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssd;
  if (a == nullptr) return SSD_ERR_INVALID;
  if (a->dtype != SSD_F32 && a->dtype != SSD_BF16) return SSD_ERR_INVALID;
  if (a->T < 0 || a->Hkv < 1 || a->num_pages < 0 || a->page_tokens < 1) return SSD_ERR_INVALID;
  if ((a->dh != 64 && a->dh != 128) || !scale_block_ok(a->scale_block) || a->Hkv > 65535) return SSD_ERR_UNSUPPORTED;
  if (a->page_tokens >= (1LL << 31) || a->num_pages >= (1LL << 31) || a->num_pages * a->page_tokens >= (1LL << 31))
    return SSD_ERR_UNSUPPORTED;
  if (a->T >= (1LL << 31)) return SSD_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(a->Hkv) * a->dh;
  if (a->k_stride < row || a->v_stride < row) return SSD_ERR_INVALID;
  if (a->T == 0) return SSD_OK;
  if (a->k_stride > (1LL << 59) / a->T || a->v_stride > (1LL << 59) / a->T) return SSD_ERR_UNSUPPORTED;
  if (!a->k_new || !a->v_new || !a->slot_map || !a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale)
    return SSD_ERR_INVALID;
  const int es = a->dtype == SSD_BF16 ? 2 : 4;
  if (!aligned(a->k_new, 16) || !aligned(a->v_new, 16) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) ||
      a->k_stride * es % 16 != 0 || a->v_stride * es % 16 != 0)
    return SSD_ERR_UNSUPPORTED;
  const int64_t codes = a->num_pages * a->page_tokens * row;
  const int64_t scales = 4 * a->num_pages * a->Hkv * ((a->page_tokens + a->scale_block - 1) / a->scale_block);
  const Span spans[] = {{a->k_cache, codes}, {a->v_cache, codes}, {a->k_scale, scales}, {a->v_scale, scales},
                        {a->k_new, ((a->T - 1) * a->k_stride + row) * es}, {a->v_new, ((a->T - 1) * a->v_stride + row) * es},
                        {a->slot_map, 4 * a->T}};
  if (overlap(spans, 4, 7)) return SSD_ERR_INVALID;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  // rows a CTA looks at: one while there are few, so that single tokens run side by side;
  // up to 128, a run for each of its groups, where most rows continue a run
  int range = 1;
  while (range < kMaxScaleBlock && a->T * a->Hkv * 2 / range > 4096) range *= 2;
  const int64_t ctas = (a->T + range - 1) / range * 2 * a->Hkv;
  if (ctas > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas));
  const cudaError_t e = by_warps(a->scale_block, [&](auto w) {
    return a->dtype == SSD_BF16
        ? launch_pdl(k_append_quant<uint16_t, w()>, grid, dim3(kQuantThreads), 0, s, *a, range, hdr)
        : launch_pdl(k_append_quant<float, w()>, grid, dim3(kQuantThreads), 0, s, *a, range, hdr);
  });
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  count_launch();
  return check_launch();
}

extern "C" int ssd_commit_kv_quant(const ssd_commit_quant_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssd;
  if (a == nullptr) return SSD_ERR_INVALID;
  if (a->dtype != SSD_F32 && a->dtype != SSD_BF16) return SSD_ERR_INVALID;
  if (a->B < 0 || a->NB < 1 || a->Dmax < 1 || a->Hkv < 1) return SSD_ERR_INVALID;
  if ((a->dh != 64 && a->dh != 128) || !scale_block_ok(a->scale_block) || a->Hkv > 65535 || a->Dmax > 256)
    return SSD_ERR_UNSUPPORTED;
  if (static_cast<double>(a->B) * a->NB * a->Dmax * a->Hkv >= 0x1p40) return SSD_ERR_UNSUPPORTED;
  int64_t page_tokens = kPageTokens;
  if (a->block_table != nullptr) {
    if (a->pages_per_seq < 1 || a->num_pages < 1) return SSD_ERR_INVALID;
    if (a->num_pages > 0x7fffffffLL / kPageTokens || a->pages_per_seq > 0x7fffffff / kPageTokens) return SSD_ERR_UNSUPPORTED;
  } else {
    if (a->P_max < 0) return SSD_ERR_INVALID;
    if (a->P_max >= (1LL << 31) || a->P_max * a->B >= (1LL << 31)) return SSD_ERR_UNSUPPORTED;
    page_tokens = a->P_max > 0 ? a->P_max : 1;
  }
  if (a->B == 0) return SSD_OK;
  if (!a->k_cand || !a->v_cand || !a->prefix_len || !a->best_blk || !a->n_out || !a->new_len) return SSD_ERR_INVALID;
  if ((a->block_table != nullptr || a->P_max > 0) && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale))
    return SSD_ERR_INVALID;
  if (!aligned(a->k_cand, 16) || !aligned(a->v_cand, 16) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16))
    return SSD_ERR_UNSUPPORTED;
  const int64_t pages = a->block_table != nullptr ? a->num_pages : a->P_max > 0 ? a->B : 0;
  const int64_t cand = static_cast<int64_t>(a->B) * a->NB * a->Dmax * a->Hkv * a->dh * (a->dtype == SSD_BF16 ? 2 : 4);
  const int64_t codes = pages * page_tokens * a->Hkv * a->dh;
  const int64_t scales = 4 * pages * a->Hkv * ((page_tokens + a->scale_block - 1) / a->scale_block);
  const Span spans[] = {{a->k_cache, codes}, {a->v_cache, codes}, {a->k_scale, scales}, {a->v_scale, scales},
                        {a->new_len, 4LL * a->B}, {a->prefix_len, 4LL * a->B}, {a->k_cand, cand}, {a->v_cand, cand},
                        {a->best_blk, 4LL * a->B}, {a->n_out, 4LL * a->B},
                        {a->block_table, 4LL * a->B * a->pages_per_seq}};
  if (overlap(spans, 5, 11)) return SSD_ERR_INVALID;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  // blocks that Dmax rows can touch
  const int segs = (a->Dmax + a->scale_block - 2) / a->scale_block + 1;
  const dim3 grid(static_cast<unsigned>(a->B), static_cast<unsigned>(a->Hkv), static_cast<unsigned>(2 * segs));
  const cudaError_t e = by_warps(a->scale_block, [&](auto w) {
    return a->dtype == SSD_BF16
        ? launch_pdl(k_commit_quant<uint16_t, w()>, grid, dim3(32 * w()), 0, s, *a, page_tokens, segs, hdr)
        : launch_pdl(k_commit_quant<float, w()>, grid, dim3(32 * w()), 0, s, *a, page_tokens, segs, hdr);
  });
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  count_launch();
  return check_launch();
}
