// Paged key/value cache: pages and slots from request lengths, and the store
// of new tokens' keys and values.
#pragma once
#include "common.h"

namespace ctcpb_lm {

// ------------------------------------------------------------------ plan --
//
// With have = ceil(len / ps), row r appends a = min(cnt, capacity - start_r)
// tokens (start: exclusive sum of cnt) and needs
//   need = min(ceil((len + a) / ps), table width) - have
// pages, which are pool[taken + off_r + k], off the exclusive sum of need.
// Token p of the row has slot table[r][p / ps] * ps + p % ps.
//
// The whole call is one launch: it moves a few bytes per token, so what it
// costs is latency.  Every workgroup scans the rows (in tiles of kPlanRows,
// one row per thread) and handles those tokens of the tile that lie in its own
// part of the slot map.  The token that opens a page writes its table entry.
constexpr int kPlanThreads = 1024;
constexpr uint32_t kPlanMost = 1u << 30;   // sums saturate here

__device__ inline uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kPlanMost); }

// Exclusive saturating sums over the workgroup's threads of v; *total gets the
// sum.  `part`: LDS, one word per wave and one more.
__device__ inline uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  uint32_t x = v;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if (lane >= d) x = sat_add(x, y);
  }
  if (lane == 63) part[wave] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    const uint32_t p = part[w];
    if (w < wave) before = sat_add(before, p);
    all = sat_add(all, p);
  }
  const uint32_t up = __shfl_up(x, 1);
  __syncthreads();   // `part` may be written again
  *total = all;
  return sat_add(before, lane ? up : 0);
}

struct PlanArgs {
  const int32_t *lengths, *counts, *pool, *taken;
  int32_t *tables, *slots, *positions, *starts, *out_lengths, *out_taken, *status;
  int64_t table_stride;
  int32_t rows, width, pool_size, page_log, capacity, per_block;
};

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  __shared__ uint32_t first[kPlanThreads + 1], off[kPlanThreads];
  __shared__ int32_t len[kPlanThreads];
  __shared__ uint32_t part[kPlanThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint32_t cap = a.capacity;
  const uint32_t ps = 1u << a.page_log;
  const uint32_t taken = min(max(*a.taken, 0), a.pool_size);
  const uint32_t lo = (uint32_t)blockIdx.x * a.per_block;
  const uint32_t hi = min(lo + (uint32_t)a.per_block, cap);
  uint32_t token_base = 0, page_base = 0;
  for (int r0 = 0; r0 < a.rows; r0 += nt) {
    const int r = r0 + tid;
    const bool in = r < a.rows;
    const uint32_t n =
        in ? (uint32_t)min((int64_t)max(a.lengths[r], 0), (int64_t)a.width << a.page_log) : 0;
    const uint32_t cnt = in ? min((uint32_t)max(a.counts[r], 0), kPlanMost) : 0;
    uint32_t sum;
    const uint32_t start = sat_add(token_base, block_scan(cnt, part, &sum));
    const uint32_t add = start < cap ? min(cnt, cap - start) : 0;
    const uint32_t have = (n + ps - 1) >> a.page_log;
    const uint32_t want = (n + add + ps - 1) >> a.page_log;
    const uint32_t need = min(want, (uint32_t)a.width) - have;
    uint32_t pages;
    const uint32_t mine = sat_add(page_base, block_scan(need, part, &pages));
    first[tid] = start;
    if (tid == nt - 1) first[nt] = sat_add(start, cnt);
    off[tid] = mine;
    len[tid] = n;
    if (blockIdx.x == 0 && in) {
      const uint32_t left = a.pool_size - taken;
      const uint32_t got = mine < left ? min(need, left - mine) : 0;
      a.starts[r] = start;
      a.out_lengths[r] = min(n + add, (have + got) << a.page_log);
      a.status[r] = (got < need ? 1 : 0) | (want > (uint32_t)a.width ? 2 : 0) | (add < cnt ? 4 : 0);
      if (r == a.rows - 1) a.starts[a.rows] = sat_add(start, cnt);
    }
    __syncthreads();
    const uint32_t end = min(hi, first[nt]);
    for (uint32_t j = max(lo, token_base) + tid; j < end; j += nt) {
      // the last row of the tile that starts at or before j (empty rows share a start)
      int s = 0;
      for (int step = kPlanThreads / 2; step; step >>= 1)
        if (s + step < nt && first[s + step] <= j) s += step;
      const uint32_t pos = (uint32_t)len[s] + (j - first[s]);
      const uint32_t p = pos >> a.page_log;
      const uint32_t held = ((uint32_t)len[s] + ps - 1) >> a.page_log;
      int32_t page = -1;
      if (p < (uint32_t)a.width) {
        int32_t* entry = a.tables + (int64_t)(r0 + s) * a.table_stride + p;
        if (p < held) {
          page = *entry;
        } else {
          const uint32_t at = taken + off[s] + (p - held);
          if (at < (uint32_t)a.pool_size) page = a.pool[at];
          if ((pos & (ps - 1)) == 0) *entry = page;
        }
      }
      a.slots[j] = page < 0 ? -1 : (int32_t)(((uint32_t)page << a.page_log) + (pos & (ps - 1)));
      a.positions[j] = pos;
    }
    token_base = sat_add(token_base, sum);
    page_base = sat_add(page_base, pages);
    __syncthreads();   // the tile's arrays are rewritten
  }
  for (uint32_t j = max(lo, token_base) + tid; j < hi; j += nt) {
    a.slots[j] = -1;
    a.positions[j] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.out_taken[0] = min(taken + page_base, (uint32_t)a.pool_size);
    if (a.rows == 0) a.starts[0] = 0;
  }
}

struct ReleaseArgs {
  const uint8_t* finished;
  const int32_t *lengths, *tables, *taken;
  int32_t *pool, *out_lengths, *out_taken;
  int64_t table_stride;
  int32_t rows, width, pool_size, page_log;
};

// One workgroup: two passes over the rows, the first to count the pages that
// come back (it fixes where the first of them goes), the second to move them,
// a wave per row.
__global__ __launch_bounds__(kPlanThreads) void release_kernel(ReleaseArgs a) {
  __shared__ uint32_t off[kPlanThreads], num[kPlanThreads], part[kPlanThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint32_t ps = 1u << a.page_log;
  const auto pages_of = [&](int r) -> uint32_t {
    if (r >= a.rows || !a.finished[r]) return 0;
    const uint32_t n =
        (uint32_t)min((int64_t)max(a.lengths[r], 0), (int64_t)a.width << a.page_log);
    return (n + ps - 1) >> a.page_log;
  };
  uint32_t total = 0;
  for (int r0 = 0; r0 < a.rows; r0 += nt) {
    uint32_t sum;
    block_scan(pages_of(r0 + tid), part, &sum);
    total = sat_add(total, sum);
  }
  const int32_t taken = min(max(*a.taken, 0), a.pool_size);
  const int32_t left = taken - (int32_t)min(total, (uint32_t)taken);
  uint32_t base = 0;
  for (int r0 = 0; r0 < a.rows; r0 += nt) {
    const int r = r0 + tid;
    const uint32_t n = pages_of(r);
    uint32_t sum;
    off[tid] = sat_add(base, block_scan(n, part, &sum));
    num[tid] = n;
    if (r < a.rows) a.out_lengths[r] = a.finished[r] ? 0 : a.lengths[r];
    __syncthreads();
    for (int w = tid >> 6; w < nt && r0 + w < a.rows; w += nt >> 6)
      for (uint32_t k = tid & 63; k < num[w]; k += 64) {
        // a row released twice asks for more pages than were taken: the rest is left out
        const uint32_t at = (uint32_t)left + off[w] + k;
        if (at < (uint32_t)taken) a.pool[at] = a.tables[(int64_t)(r0 + w) * a.table_stride + k];
      }
    base = sat_add(base, sum);
    __syncthreads();
  }
  if (tid == 0) a.out_taken[0] = left;
}

// ----------------------------------------------------------------- store --
struct CacheView {
  char* data;
  int64_t page, token, head;   // strides in bytes
};

struct StoreArgs {
  const char *k, *v;
  int64_t k_t, k_h, v_t, v_h;   // strides in bytes
  const int32_t* slots;
  CacheView kc, vc;
  int64_t pieces;               // tokens * heads * pieces per head
  int32_t heads, per_head;      // pieces (of sizeof(Piece) bytes) per head
  int32_t page_log, num_slots;
};

// A copy: bound by memory, 2 x (read + write) of the tokens' rows.  A thread
// moves the same piece of the key and of the value, so that a token's slot is
// looked up once for both.
template <typename Piece>
__global__ __launch_bounds__(256) void store_kernel(StoreArgs a) {
  const int64_t step = (int64_t)gridDim.x * 256;
  const int32_t row = a.heads * a.per_head;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.pieces; i += step) {
    const int32_t t = (int32_t)(i / row), rest = (int32_t)(i % row);
    const int32_t slot = a.slots[t];
    if ((uint32_t)slot >= (uint32_t)a.num_slots) continue;
    const int32_t h = rest / a.per_head, p = rest % a.per_head;
    const int64_t page = slot >> a.page_log, at = slot & ((1 << a.page_log) - 1);
    const int64_t b = (int64_t)p * sizeof(Piece);
    const Piece kv = *reinterpret_cast<const Piece*>(a.k + t * a.k_t + h * a.k_h + b);
    const Piece vv = *reinterpret_cast<const Piece*>(a.v + t * a.v_t + h * a.v_h + b);
    *reinterpret_cast<Piece*>(a.kc.data + page * a.kc.page + at * a.kc.token + h * a.kc.head + b) =
        kv;
    *reinterpret_cast<Piece*>(a.vc.data + page * a.vc.page + at * a.vc.token + h * a.vc.head + b) =
        vv;
  }
}

}  // namespace ctcpb_lm
