// Attention over the 8-bit cache: argument checks, and the kernel for few packed rows
// (single tokens, short chains; any group size and head dim 64 or 128).
//
// Mathematics. With codes c, block scales sk and sv, and y_j = scale log2e (q.c_j) sk_j +
// log2 sv_j, the output is  sum_j 2^(y_j - M) c_j / sum_j 2^(y_j - M) / sv_j  for any M:
// the values' scale rides in the exponent, so no element is multiplied by it, and the
// denominator gets one multiplication by 1/sv for each group of keys of one block. M is
// the running maximum of y, moved only when it grows by more than 2^8.
//
// What bounds it: the cache's bytes, read once (2 dh bytes a key and kv head). A warp
// takes 16 keys a step and keeps its own running maximum, sum and output (online
// softmax), so warps share nothing until the end. Each lane copies exactly the bytes that
// its own matrix fragments need (cp.async, 16 bytes, whole 32-byte sectors) into a private
// ring in shared memory several steps ahead and reads them back itself: no barrier, no
// transpose. That works because both products may permute their inner index: for Q K^T
// lane (g, t) holds elements 16t .. 16t+15 of each 64-element half of key g, and Q is laid
// out alike; for P V it holds, for its four keys, the output elements dh/8 g .. (columns
// permuted alike on the way out). Codes become fp16 exactly by one conversion for two; q is
// scaled by a power of two per row to fit fp16, probabilities are rounded to fp16 (at most
// 2^8). mma.sync is enough here: 16 packed rows are an eighth of the smallest tcgen05
// tile, and the matrix work is under half of the time the bytes take.
//
// The CTAs of a cluster split the steps of a (sequence, kv head) evenly by its own length;
// rank 0 adds the own-block keys (bf16 products, probabilities as a sum of two bf16). Warps
// and then CTAs merge maxima, sums and outputs in a fixed order through shared memory.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "ssd_attn_quant.cuh"
#include "ssd_tc.cuh"

namespace ssd {

constexpr int kRowsWarps = 8;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kStepKeys = 16;
constexpr int kRowsTile = 16;             // packed rows of a CTA
constexpr int kRowsStages = 3;

template <int DH>
struct RowsSmem {
  static constexpr int kStep = 2 * kStepKeys * DH + 32;      // K and V bytes of a step, then two scales
  static constexpr int kRing = kRowsWarps * kRowsStages * kStep;
  static constexpr int kPart = kRowsWarps * kRowsTile * DH * 4;   // warps' outputs, over the ring
  static constexpr int kMain = kRing > kPart ? kRing : kPart;
  static constexpr int kQ = kRowsTile * DH * 2;              // fp16 fragments
  static constexpr int kOut = kRowsTile * DH * 4;            // the CTA's merged output
  static constexpr int kStat = (kRowsWarps + 1) * kRowsTile * 2 * 4;   // maxima and sums
  static constexpr int kBytes = kMain + kQ + kOut + kStat;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_b16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// `n` bytes (16, 8 or 4) of global memory to shared memory, zeros when !take
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool take) {
  const int n = take ? N : 0;
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}

__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// a running softmax of two rows (g and g + 8) of a warp's fragment
struct RunningRows {
  float m[2], l[2];
};

// The running maximum after 16 keys with scores y (log2 units; -inf where masked), the
// factor on what was summed before, and whether any lane of the warp needs it.
__device__ __forceinline__ bool move_max(RunningRows& r, const float (&y)[2][4], float (&ref)[2], float (&alpha)[2]) {
  bool moved = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float top = quad_max(fmaxf(fmaxf(y[0][2 * i], y[0][2 * i + 1]), fmaxf(y[1][2 * i], y[1][2 * i + 1])));
    alpha[i] = 1.f;
    if (top > r.m[i] + 8.f) {             // also the first keys: m is -inf
      alpha[i] = ex2_approx(r.m[i] - top);
      r.m[i] = top;
      moved = true;
    }
    ref[i] = r.m[i] == -INFINITY ? 0.f : r.m[i];
  }
  return __any_sync(0xffffffffu, moved);
}

template <int DH>
__global__ void __launch_bounds__(kRowsThreads, 2)
k_attn_quant_rows(AttnQuantParams p) {
  using SM = RowsSmem<DH>;
  constexpr int KS = DH / 16;             // inner steps of Q K^T, and 8-column pairs of the output
  constexpr int NV = DH / 8;              // output tiles of 8 columns
  constexpr int EV = DH / 8;              // code bytes of a value row that a lane takes
  constexpr int KC = DH / 64;             // 16-byte chunks of a key row that a lane takes
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring = smem;
  uint32_t* qs = reinterpret_cast<uint32_t*>(smem + SM::kMain);
  float* merged = reinterpret_cast<float*>(smem + SM::kMain + SM::kQ);
  float* stat_m = merged + kRowsTile * DH;                    // [warps + 1][rows]
  float* stat_l = stat_m + (kRowsWarps + 1) * kRowsTile;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t rank, S;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(S));
  const int bk = blockIdx.x / S;
  const int b = bk / p.Hkv, kvh = bk % p.Hkv;
  const int G = p.Hq / p.Hkv, NT = p.NB * p.Dmax;
  const int r0 = blockIdx.y * kRowsTile, rows = min(kRowsTile, NT * G - r0);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // present rows of the tile; the CTAs of a cluster hold the same rows and leave together
  bool here = false;
  if (tid < rows) {
    const int tt = (r0 + tid) / G;
    here = tt % p.Dmax < p.blk_len[b * p.NB + tt / p.Dmax];
  }
  if (!__syncthreads_or(here)) return;

  int64_t P = p.prefix_len[b];
  if (P < 0 || P > p.capacity) {
    if (tid == 0) record_error(p.hdr, SSD_ERR_DEVICE, 440);
    P = 0;
  }
  const int steps = static_cast<int>((P + kStepKeys - 1) / kStepKeys);
  const int step0 = static_cast<int>(static_cast<int64_t>(steps) * rank / S) + warp;
  const int step1 = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / S);

  // ---- the ring: copies of step s into stage i (an empty group past the end)
  const int pt_log2 = 7;
  auto page_of = [&](int s) -> int64_t {                // page of a step; a contiguous cache's is the sequence
    if (p.block_table == nullptr || s >= step1) return b;
    return p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + ((s * kStepKeys) >> pt_log2)];
  };
  uint8_t* my = ring + warp * kRowsStages * SM::kStep;
  auto issue = [&](int s, int stage, int64_t page) {
    if (s < step1) {
      const int64_t key0 = static_cast<int64_t>(s) * kStepKeys;
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) record_error(p.hdr, SSD_ERR_DEVICE, 441);
        page = 0;
      }
      const int64_t place = p.block_table == nullptr ? key0 : key0 & (kPageTokens - 1);
      const int64_t ph = page * p.Hkv + kvh;
      const int64_t at = (ph * p.page_tokens + place) * DH;
      const int left = static_cast<int>(P - key0);         // keys of the step that exist
      const uint32_t dst = tc::smem_u32(my + stage * SM::kStep) + lane * 16;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < KC; ++c)
          copy_async<16>(dst + (n * KC + c) * 512, p.k_cache + at + (n * 8 + g < left ? (n * 8 + g) * DH + c * 64 + t4 * 16 : 0),
                         n * 8 + g < left);
      const uint32_t dv = tc::smem_u32(my + stage * SM::kStep) + kStepKeys * DH + lane * EV;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = 2 * t4 + (j & 1) + (j >> 1) * 8;
        copy_async<EV>(dv + j * 32 * EV, p.v_cache + at + (key < left ? key * DH + g * EV : 0), key < left);
      }
      if (lane < 2) {
        const float* sc = (lane == 0 ? p.k_scale : p.v_scale) + ph * p.blocks + (place >> p.sb_log2);
        copy_async<4>(tc::smem_u32(my + stage * SM::kStep) + 2 * kStepKeys * DH + lane * 4, sc, true);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t next_page = page_of(step0);
#pragma unroll
  for (int i = 0; i < kRowsStages - 1; ++i) {
    issue(step0 + i * kRowsWarps, i, next_page);
    next_page = page_of(step0 + (i + 1) * kRowsWarps);
  }

  // ---- Q: a power of two per row brings the largest magnitude into [1, 2); fp16 fragments
  // in shared memory, [inner step][lane][4 words]
  {
    // thread = (row, 16 lanes of DH/16 elements)
    const int row = tid >> 4, part = tid & 15;
    constexpr int E = DH / 16;
    float x[E];
    const int rr = r0 + row;
    const bool ok = row < rows;
    const uint16_t* src = p.q + ((static_cast<int64_t>(b) * NT + rr / G) * p.Hq + kvh * G + rr % G) * DH + part * E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = ok ? bf16_to_f32(src[e]) : 0.f;
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int ex = static_cast<int>(__float_as_uint(m) >> 23);     // biased exponent; 0 and 255 stay unscaled
    const bool sc = ex > 0 && ex < 254;
    const float mul = sc ? __uint_as_float(static_cast<uint32_t>(254 - ex) << 23) : 1.f;
    if (part == 0) stat_m[row] = sc ? __uint_as_float(static_cast<uint32_t>(ex) << 23) : 1.f;
    // element d of a row: half c = d / 64, lane t = d % 64 / 16, inner step 4c + d % 16 / 4,
    // words a0/a1 (first pair of the four) or a2/a3 (second pair); rows 8.. are a1, a3
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const int d = part * E + e;
      const int ks = (d >> 6) * 4 + ((d & 15) >> 2), t = (d & 63) >> 4, word = ((d >> 1) & 1) * 2 + (row >> 3);
      qs[(ks * 32 + (row & 7) * 4 + t) * 4 + word] = pack_f16(x[e] * mul, x[e + 1] * mul);
    }
  }
  __syncthreads();
  float q_mul[2];
  q_mul[0] = stat_m[g] * p.scale_log2;
  q_mul[1] = stat_m[g + 8] * p.scale_log2;
  __syncthreads();                                   // stat_m is reused below

  RunningRows run;
  run.m[0] = run.m[1] = -INFINITY;
  run.l[0] = run.l[1] = 0.f;
  float o[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;

  auto rescale = [&](const float (&alpha)[2]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      o[j][0] *= alpha[0];
      o[j][1] *= alpha[0];
      o[j][2] *= alpha[1];
      o[j][3] *= alpha[1];
    }
    run.l[0] *= alpha[0];
    run.l[1] *= alpha[1];
  };

  // ---- own-block keys (rank 0), 16 slots a step from the block of the tile's first row
  if (rank == 0) {
    const int t_first = r0 / G, t_last = (r0 + rows - 1) / G;
    const int s_base = t_first / p.Dmax * p.Dmax;
    const int lim = t_last + 1 - s_base;
    int tr[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      tr[i] = r < rows ? (r0 + r) / G : -1;            // slot of the row; none is allowed for rows past the end
      lo[i] = r < rows ? tr[i] / p.Dmax * p.Dmax : 0;
    }
    for (int s = warp; s * kStepKeys < lim; s += kRowsWarps) {
      const int slot0 = s_base + s * kStepKeys;
      float c[2][4] = {};
      // inner step ks: elements 16 ks + 4 t4 .. + 3 of a row
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 v = make_uint2(0u, 0u);
          if (g + 8 * i < rows) {
            const int rr = r0 + g + 8 * i;
            v = *reinterpret_cast<const uint2*>(
                p.q + ((static_cast<int64_t>(b) * NT + rr / G) * p.Hq + kvh * G + rr % G) * DH + ks * 16 + t4 * 4);
          }
          a[i] = v.x;
          a[2 + i] = v.y;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int slot = slot0 + n * 8 + g;
          uint2 v = make_uint2(0u, 0u);
          if (slot <= t_last)
            v = *reinterpret_cast<const uint2*>(p.k_cand + ((static_cast<int64_t>(b) * NT + slot) * p.Hkv + kvh) * DH +
                                                ks * 16 + t4 * 4);
          mma_b16(c[n], a, v.x, v.y);
        }
      }
      float y[2][4], ref[2], alpha[2];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int slot = slot0 + n * 8 + 2 * t4 + (e & 1);
          const int i = e >> 1;
          y[n][e] = slot >= lo[i] && slot <= tr[i] ? c[n][e] * p.scale_log2 : -INFINITY;
        }
      if (move_max(run, y, ref, alpha)) rescale(alpha);
      uint32_t hi[4], low[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float w0 = ex2_approx(y[n][2 * i] - ref[i]), w1 = ex2_approx(y[n][2 * i + 1] - ref[i]);
          run.l[i] += w0 + w1;
          const uint32_t h = tc::pack_bf16(w0, w1);
          hi[2 * n + i] = h;
          low[2 * n + i] = tc::pack_bf16(w0 - __uint_as_float(h << 16), w1 - __uint_as_float(h & 0xffff0000u));
        }
      // values: lane's keys 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9; columns g * EV + j
      uint32_t v[4][EV / 2];
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
      bool odd_value = false;                          // an infinity or NaN
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int u = 0; u < EV / 2; ++u)
          odd_value |= (v[k][u] & 0x7f800000u) == 0x7f800000u || (v[k][u] & 0x7f80u) == 0x7f80u;
      if (!__any_sync(0xffffffffu, odd_value)) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(v[0][j / 2], v[1][j / 2], sel), b1 = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
          mma_b16(o[j], hi, b0, b1);
          mma_b16(o[j], low, b0, b1);
        }
      } else {
        // slots of other blocks and of absent tokens may hold anything, and 0 * inf is not 0:
        // key by key, for the rows that see it
#pragma unroll 1
        for (int k = 0; k < kStepKeys && slot0 + k <= t_last; ++k) {
          const int from = (lane & ~3) | ((k & 7) >> 1);
          float yk[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float first = k < 8 ? y[0][2 * i] : y[1][2 * i], second = k < 8 ? y[0][2 * i + 1] : y[1][2 * i + 1];
            yk[i] = __shfl_sync(0xffffffffu, (k & 1) ? second : first, from);
          }
          const uint16_t* src = p.v_cand + ((static_cast<int64_t>(b) * NT + slot0 + k) * p.Hkv + kvh) * DH;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (slot0 + k < lo[i] || slot0 + k > tr[i]) continue;
            const float w = ex2_approx(yk[i] - ref[i]);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                o[j][2 * i + h] = fmaf(w, bf16_to_f32(src[EV * (2 * t4 + h) + j]), o[j][2 * i + h]);
          }
        }
      }
    }
  }

  // ---- prefix keys
  int stage = 0;
  for (int s = step0; s < step1; s += kRowsWarps) {
    {
      const int ahead = s + (kRowsStages - 1) * kRowsWarps;
      const int into = stage == 0 ? kRowsStages - 1 : stage - 1;
      __syncwarp();                                  // the scales in that stage have been read
      issue(ahead, into, next_page);
      next_page = page_of(ahead + kRowsWarps);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kRowsStages - 1) : "memory");
    __syncwarp();                                    // the scales are another lane's copies
    const uint8_t* st = my + stage * SM::kStep;
    stage = stage + 1 == kRowsStages ? 0 : stage + 1;
    const float2 sc = *reinterpret_cast<const float2*>(st + 2 * kStepKeys * DH);
    float c[2][4] = {};
#pragma unroll
    for (int ch = 0; ch < KC; ++ch) {
      const uint4 k0 = *reinterpret_cast<const uint4*>(st + ch * 512 + lane * 16);
      const uint4 k1 = *reinterpret_cast<const uint4*>(st + (KC + ch) * 512 + lane * 16);
      const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 aq = *reinterpret_cast<const uint4*>(qs + ((ch * 4 + i) * 32 + lane) * 4);
        const uint32_t a[4] = {aq.x, aq.y, aq.z, aq.w};
        mma_f16(c[0], a, e4m3x2_to_f16x2(w0[i]), e4m3x2_to_f16x2(w0[i] >> 16));
        mma_f16(c[1], a, e4m3x2_to_f16x2(w1[i]), e4m3x2_to_f16x2(w1[i] >> 16));
      }
    }
    const int left = static_cast<int>(P - static_cast<int64_t>(s) * kStepKeys);
    const float lv = fmaxf(__log2f(sc.y), kLeastVScaleLog2);
    float y[2][4], ref[2], alpha[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = fmaf(c[n][e], q_mul[e >> 1] * sc.x, lv);
        y[n][e] = n * 8 + 2 * t4 + (e & 1) < left ? v : -INFINITY;
      }
    if (move_max(run, y, ref, alpha)) rescale(alpha);
    const float inv_sv = ex2_approx(-lv);
    uint32_t a[4];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float w0 = ex2_approx(y[n][2 * i] - ref[i]), w1 = ex2_approx(y[n][2 * i + 1] - ref[i]);
        sum[i] += w0 + w1;
        a[2 * n + i] = pack_f16(w0, w1);
      }
    run.l[0] = fmaf(sum[0], inv_sv, run.l[0]);
    run.l[1] = fmaf(sum[1], inv_sv, run.l[1]);
    uint32_t v[4][EV / 4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint8_t* src = st + kStepKeys * DH + k * 32 * EV + lane * EV;
      if constexpr (EV == 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(src);
        v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(src);
        v[k][0] = x.x; v[k][1] = x.y;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; j += 2) {
      // bytes j, j + 1 of two keys side by side: one pair of codes for each column
      const uint32_t sel = (j & 2) ? 0x7362u : 0x5140u;
      const uint32_t c0 = __byte_perm(v[0][j / 4], v[1][j / 4], sel), c1 = __byte_perm(v[2][j / 4], v[3][j / 4], sel);
      mma_f16(o[j], a, e4m3x2_to_f16x2(c0), e4m3x2_to_f16x2(c1));
      mma_f16(o[j + 1], a, e4m3x2_to_f16x2(c0 >> 16), e4m3x2_to_f16x2(c1 >> 16));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // ---- merge the warps
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float l = run.l[i];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t4 == 0) {
      stat_m[warp * kRowsTile + g + 8 * i] = run.m[i];
      stat_l[warp * kRowsTile + g + 8 * i] = l;
    }
  }
  __syncthreads();                                   // also: every ring is idle
  float* part = reinterpret_cast<float*>(ring);      // [warp][row][DH]
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, stat_m[w * kRowsTile + r]);
    const float f = run.m[i] == -INFINITY ? (run.l[i] == 0.f ? 0.f : 1.f) : ex2_approx(run.m[i] - M);
    float* dst = part + (warp * kRowsTile + r) * DH;
    // tile j, columns 2 t4 and 2 t4 + 1 stand for elements EV (2 t4) + j and EV (2 t4 + 1) + j
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NV; j += 4)
        *reinterpret_cast<float4*>(dst + EV * (2 * t4 + h) + j) =
            make_float4(o[j][2 * i + h] * f, o[j + 1][2 * i + h] * f, o[j + 2][2 * i + h] * f, o[j + 3][2 * i + h] * f);
  }
  if (tid < kRowsTile) {
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, stat_m[w * kRowsTile + tid]);
    for (int w = 0; w < kRowsWarps; ++w) {
      const float m = stat_m[w * kRowsTile + tid], l = stat_l[w * kRowsTile + tid];
      L += m == -INFINITY ? l : l * ex2_approx(m - M);        // no key: l is 0 (or NaN, which stays)
    }
    stat_m[kRowsWarps * kRowsTile + tid] = M;
    stat_l[kRowsWarps * kRowsTile + tid] = L;
  }
  __syncthreads();
  for (int e = tid; e < rows * DH; e += kRowsThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) v += part[w * kRowsTile * DH + e];
    merged[e] = v;
  }
  // ---- merge the CTAs of the cluster: each takes a share of the elements
  if (S > 1) tc::cluster_sync(); else __syncthreads();
  const uint32_t sm = tc::smem_u32(stat_m + kRowsWarps * kRowsTile), sl = tc::smem_u32(stat_l + kRowsWarps * kRowsTile),
                 so = tc::smem_u32(merged);
  for (int e = static_cast<int>(rank) * kRowsThreads + tid; e < rows * DH; e += static_cast<int>(S) * kRowsThreads) {
    const int row = e / DH;
    const int rr = r0 + row, tt = rr / G;
    float v, L;
    if (S == 1) {
      v = merged[e];
      L = stat_l[kRowsWarps * kRowsTile + row];
    } else {
      float M = -INFINITY;
      for (uint32_t c = 0; c < S; ++c) M = fmaxf(M, ld_peer(tc::map_peer(sm + row * 4, c)));
      v = 0.f;
      L = 0.f;
      for (uint32_t c = 0; c < S; ++c) {
        const float m = ld_peer(tc::map_peer(sm + row * 4, c));
        const float f = m == -INFINITY ? 1.f : ex2_approx(m - M);
        L = fmaf(ld_peer(tc::map_peer(sl + row * 4, c)), f, L);
        v = fmaf(ld_peer(tc::map_peer(so + e * 4, c)), f, v);
      }
    }
    if (tt % p.Dmax < p.blk_len[b * p.NB + tt / p.Dmax]) {
      const int64_t at = ((static_cast<int64_t>(b) * NT + tt) * p.Hq + kvh * G + rr % G) * DH + e % DH;
      const float out = v / L;
      if (p.out_f32) static_cast<float*>(p.out)[at] = out;
      else {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(out));
        static_cast<uint16_t*>(p.out)[at] = h;
      }
    }
  }
  if (S > 1) tc::cluster_sync();                     // a CTA's shared memory outlives its readers
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
  const int64_t tokens = a->block_table != nullptr ? a->num_pages * kPageTokens : a->B * a->P_max;
  const Span spans[] = {{a->out, rows * (a->out_dtype == SSD_F32 ? 4 : 2)}, {a->q, 2 * rows}, {a->k_cand, cand},
                        {a->v_cand, cand}, {a->k_cache, tokens * a->Hkv * a->dh}, {a->v_cache, tokens * a->Hkv * a->dh}};
  if (overlap(spans, 1, 6)) return SSD_ERR_INVALID;
  return SSD_OK;
}

template <int DH>
static int rows_launch(const AttnQuantParams& p, int mtiles, cudaStream_t s) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return SSD_ERR_CUDA;
  std::call_once(once[dev], [dev] {
    err[dev] = cudaFuncSetAttribute(k_attn_quant_rows<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, RowsSmem<DH>::kBytes);
  });
  if (err[dev] != cudaSuccess) return SSD_ERR_CUDA;
  // CTAs that split a sequence: enough to fill the GPU several times over (their lengths
  // differ), no more than one for each 128 keys of the longest sequence the cache can hold
  const long long groups = static_cast<long long>(p.B) * p.Hkv * mtiles;
  const long long most = std::max<long long>(1, (p.capacity + 127) / 128);
  int S = 1;
  while (S < 8 && S * 2 <= most && groups * S < 4 * 304) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(p.B) * p.Hkv * S), static_cast<unsigned>(mtiles), 1);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = RowsSmem<DH>::kBytes;
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
  if (cudaLaunchKernelEx(&cfg, k_attn_quant_rows<DH>, p) != cudaSuccess) {
    cudaGetLastError();
    return SSD_ERR_CUDA;
  }
  count_launch();
  return check_launch();
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
  const int mtiles = (rows + kRowsTile - 1) / kRowsTile;
  KernelTimer timer(SSD_KERNEL_VERIFY_ATTN, s);
  return a->dh == 128 ? rows_launch<128>(p, mtiles, s) : rows_launch<64>(p, mtiles, s);
}
