// Block tables and slot maps from request lengths (Speculative Decoding 해부 page, §6:
// a pool of pages that sequences take and give back).
//
// k_page_plan, one CTA: for chunks of 1024 sequences, one thread a sequence computes how
// many pages it gives back or lacks; block scans of those counts give every page its
// place on the stack, and the pages themselves (a prompt takes hundreds, a decoding step
// one now and then) are then moved by all threads, each finding its sequence by a binary
// search in the scan. Two passes over the batch, because the trimmed pages of all
// sequences are on the stack before the first one is taken. The call is bound by latency:
// it reads 12 bytes a sequence. Taking the pages of a step of 64 sequences and trimming them
// behind it are two launches, 9.9 us replayed from a graph; admitting 512 prompts (a million
// slots, 8 400 pages) and ending them 26 us, most of it the chain of two loads a page that one
// CTA's threads keep four of on the way.
// k_slot_map: one thread for four slots, the first one's sequence by a binary search in
// row_start. Short maps are written by the plan kernel itself.
#include "ssd_kvq.cuh"

namespace ssd {

constexpr int kPlanThreads = 1024;
constexpr int kMoves = 4;         // pages a thread has on the way at once

struct SeqNeed {
  int64_t want;     // pages for cur + add tokens
  int held;
  bool ok;
};

__device__ __forceinline__ SeqNeed seq_need(const ssd_pages_args& a, int b, int held) {
  const int64_t cur = a.cur_len[b], add = a.add_len[b];
  SeqNeed n;
  n.want = (cur + add + kPageTokens - 1) / kPageTokens;
  n.held = held;
  n.ok = cur >= 0 && add >= 0 && n.want <= a.pages_per_seq && held >= 0 && held <= a.pages_per_seq;
  return n;
}

// exclusive sum over the CTA; *total gets the sum. `part` holds one value a warp.
__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                       // `part` may still be read from the call before
  if (lane == 31) part[wid] = x;
  __syncthreads();
  if (wid == 0) {
    int64_t p = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  *total = part[31];
  return x - v + (wid > 0 ? part[wid - 1] : 0);
}

// the last i in [0, n) with off[i] <= q (off ascending, off[0] <= q)
template <typename T>
__device__ __forceinline__ int last_not_above(const T* off, int n, T q) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= q) lo = mid; else hi = mid;
  }
  return lo;
}

// slots of rows t .. t + 3, of which those below slot_cap are written; `start` = row_start
__device__ __forceinline__ void fill_four(const ssd_pages_args& a, const int32_t* start, int64_t t, WsHeader* hdr) {
  int32_t out[4] = {-1, -1, -1, -1};
  const int64_t total = a.B > 0 ? start[a.B] : 0;
  if (t < total) {
    int b = last_not_above(start, a.B, static_cast<int32_t>(t));
    int64_t begin = -1, end = -1;
    const int32_t* table = nullptr;
    bool served = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (t + e >= total) break;
      if (t + e >= end) {                        // the first row, or the first one of another sequence
        while (t + e >= start[b + 1]) ++b;
        end = start[b + 1];
        begin = static_cast<int64_t>(a.cur_len[b]) - start[b];
        table = a.block_table + static_cast<int64_t>(b) * a.pages_per_seq;
        const SeqNeed n = seq_need(a, b, a.n_pages[b]);
        served = n.ok && n.held >= n.want;
      }
      if (!served) continue;
      const int64_t pos = begin + t + e;
      if (!in_range(pos / kPageTokens, a.pages_per_seq, hdr, 411)) continue;
      const int32_t page = table[pos / kPageTokens];
      if (page < 0 || page >= a.num_pages) record_error(hdr, SSD_ERR_DEVICE, 410);
      else out[e] = page * kPageTokens + static_cast<int32_t>(pos % kPageTokens);
    }
  }
  if (t + 4 <= a.slot_cap && (reinterpret_cast<uintptr_t>(a.slot_map) & 15) == 0) {
    *reinterpret_cast<int4*>(a.slot_map + t) = make_int4(out[0], out[1], out[2], out[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (t + e < a.slot_cap) a.slot_map[t + e] = out[e];
  }
}

__global__ void __launch_bounds__(kPlanThreads)
k_page_plan(ssd_pages_args a, int fill_slots, WsHeader* hdr) {
  __shared__ int64_t part[32];
  __shared__ int32_t off[kPlanThreads];
  __shared__ int32_t base[kPlanThreads];      // first page index moved
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  int64_t free0 = a.n_free[0];
  if (free0 < 0 || free0 > a.num_pages) {
    if (tid == 0) record_error(hdr, SSD_ERR_DEVICE, 400);
    free0 = free0 < 0 ? 0 : a.num_pages;
  }
  // ---- trim: pages past `want` go on the stack
  int64_t avail = free0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int trim = 0, want = 0;
    if (b < a.B) {
      const SeqNeed n = seq_need(a, b, a.n_pages[b]);
      if (!n.ok) record_error(hdr, SSD_ERR_DEVICE, 401);
      else if (n.held > n.want) {
        trim = n.held - static_cast<int>(n.want);
        want = static_cast<int>(n.want);
      }
    }
    int64_t total;
    const int64_t at = block_exclusive(trim, part, &total);
    if (total > 0) {
      off[tid] = static_cast<int32_t>(at);
      base[tid] = want;
      __syncthreads();
      for (int64_t q0 = tid; q0 < total; q0 += kMoves * kPlanThreads) {
        int32_t* entry[kMoves];
        int32_t page[kMoves];
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
          const int64_t q = q0 + u * kPlanThreads;
          if (q < total) {
            const int i = last_not_above(off, kPlanThreads, static_cast<int32_t>(q));
            entry[u] = nullptr;
            if (!in_range(b0 + i, a.B, hdr, 405) || !in_range(base[i] + (q - off[i]), a.pages_per_seq, hdr, 405)) continue;
            entry[u] = a.block_table + static_cast<int64_t>(b0 + i) * a.pages_per_seq + base[i] + (q - off[i]);
            page[u] = *entry[u];
          }
        }
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
          const int64_t q = q0 + u * kPlanThreads;
          if (q < total && (!SSD_CHECKS || entry[u] != nullptr)) {
            if (avail + q < a.num_pages) a.free_pages[avail + q] = page[u];
            else record_error(hdr, SSD_ERR_DEVICE, 402);
            *entry[u] = -1;
          }
        }
      }
      if (trim > 0) a.n_pages[b] = want;
    }
    avail += total;
  }
  if (avail > a.num_pages) avail = a.num_pages;
  __syncthreads();                            // the stack holds the trimmed pages
  // ---- grow: pages from the top of the stack, in order of b
  int64_t lacked = 0, taken = 0, rows = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int64_t grow = 0, add = 0;
    int held = 0;
    bool ok = false;
    if (b < a.B) {
      held = a.n_pages[b];
      const SeqNeed n = seq_need(a, b, held);
      ok = n.ok;
      add = max(0, a.add_len[b]);
      if (ok && n.want > held) grow = n.want - held;
    }
    int64_t total, rows_total;
    const int64_t at = block_exclusive(grow, part, &total);
    const int64_t row = block_exclusive(add, part, &rows_total);
    const bool serve = ok && (grow == 0 || lacked + at + grow <= avail);
    if (b < a.B) {
      const int64_t r = rows + row;
      a.row_start[b] = static_cast<int32_t>(r > 0x7fffffffLL ? 0x7fffffffLL : r);
      if (a.served != nullptr) a.served[b] = serve ? 1 : 0;
    }
    // the served ones of this chunk are those up to a point: the pages they take are the
    // first `take` of the chunk's
    int64_t take;
    block_exclusive(serve ? grow : 0, part, &take);
    if (take > 0) {
      off[tid] = static_cast<int32_t>(at);
      base[tid] = held;
      __syncthreads();
      for (int64_t q0 = tid; q0 < take; q0 += kMoves * kPlanThreads) {
        int32_t* entry[kMoves];
        int32_t page[kMoves];
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
          const int64_t q = q0 + u * kPlanThreads;
          if (q < take) {
            entry[u] = nullptr;
            if (!in_range(avail - 1 - (lacked + q), a.num_pages, hdr, 406)) continue;
            page[u] = a.free_pages[avail - 1 - (lacked + q)];
            const int i = last_not_above(off, kPlanThreads, static_cast<int32_t>(q));
            if (!in_range(b0 + i, a.B, hdr, 407) || !in_range(base[i] + (q - off[i]), a.pages_per_seq, hdr, 407)) continue;
            entry[u] = a.block_table + static_cast<int64_t>(b0 + i) * a.pages_per_seq + base[i] + (q - off[i]);
          }
        }
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
          if (q0 + u * kPlanThreads < take && (!SSD_CHECKS || entry[u] != nullptr)) {
            if (page[u] < 0 || page[u] >= a.num_pages) record_error(hdr, SSD_ERR_DEVICE, 403);
            *entry[u] = page[u];
          }
        }
      }
      if (serve && grow > 0) a.n_pages[b] = static_cast<int32_t>(held + grow);
    }
    lacked += total;
    taken += take;
    rows += rows_total;
  }
  if (tid == 0) {
    a.row_start[a.B] = static_cast<int32_t>(rows > 0x7fffffffLL ? 0x7fffffffLL : rows);
    a.n_free[0] = static_cast<int32_t>(avail - taken);
    if (rows > a.slot_cap || rows > 0x7fffffffLL) record_error(hdr, SSD_ERR_DEVICE, 404);
  }
  if (fill_slots) {
    __syncthreads();                          // tables and row_start are written
    for (int64_t t = 4 * tid; t < a.slot_cap; t += 4 * kPlanThreads) fill_four(a, a.row_start, t, hdr);
  }
}

constexpr int kSlotThreads = 256;

__global__ void __launch_bounds__(kSlotThreads)
k_slot_map(ssd_pages_args a, WsHeader* hdr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = 4 * (static_cast<int64_t>(blockIdx.x) * kSlotThreads + threadIdx.x);
  if (t < a.slot_cap) fill_four(a, a.row_start, t, hdr);
}

}  // namespace ssd

extern "C" int ssd_page_tables(const ssd_pages_args* a, void* ws, size_t ws_bytes, void* stream) {
  using namespace ssd;
  if (a == nullptr) return SSD_ERR_INVALID;
  if (a->B < 0 || a->pages_per_seq < 0 || a->num_pages < 0 || a->slot_cap < 0) return SSD_ERR_INVALID;
  if (!a->n_free || !a->row_start) return SSD_ERR_INVALID;
  if ((a->slot_map == nullptr) != (a->slot_cap == 0)) return SSD_ERR_INVALID;
  if (a->B > 0 && (!a->cur_len || !a->add_len || !a->n_pages)) return SSD_ERR_INVALID;
  if (a->B > 0 && a->pages_per_seq > 0 && !a->block_table) return SSD_ERR_INVALID;
  if (a->num_pages > 0 && !a->free_pages) return SSD_ERR_INVALID;
  if (a->num_pages > (0x7fffffffLL / kPageTokens) || a->slot_cap > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
  // the pages of 1024 sequences are counted in 32 bits
  if (a->pages_per_seq > (1 << 20)) return SSD_ERR_UNSUPPORTED;
  const Span spans[] = {{a->n_pages, 4LL * a->B}, {a->block_table, 4LL * a->B * a->pages_per_seq},
                        {a->free_pages, 4 * a->num_pages}, {a->n_free, 4}, {a->row_start, 4LL * a->B + 4},
                        {a->slot_map, 4 * a->slot_cap}, {a->served, 4LL * a->B}, {a->cur_len, 4LL * a->B},
                        {a->add_len, 4LL * a->B}};
  if (overlap(spans, 7, 9)) return SSD_ERR_INVALID;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  WsHeader* hdr = static_cast<WsHeader*>(ws);
  const int fill = a->slot_cap <= 4 * kPlanThreads ? 1 : 0;
  if (launch_pdl(k_page_plan, dim3(1), dim3(kPlanThreads), 0, s, *a, fill, hdr) != cudaSuccess) return SSD_ERR_CUDA;
  count_launch();
  if (!fill) {
    const unsigned g = static_cast<unsigned>((a->slot_cap + 4 * kSlotThreads - 1) / (4 * kSlotThreads));
    if (launch_pdl(k_slot_map, dim3(g), dim3(kSlotThreads), 0, s, *a, hdr) != cudaSuccess) return SSD_ERR_CUDA;
    count_launch();
  }
  return check_launch();
}
