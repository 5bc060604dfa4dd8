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
// costs is latency.  Every workgroup scans the rows (in tiles of ITEMS rows per
// thread, normally one tile) and handles those tokens of the tile that lie in its
// own part of the slot map.  The token that opens a page writes its table entry.
// 256 rows of one new token: 5 us on the GPU.  4096 rows of 0..512 new tokens: 18.6 us
// with a row per thread and two scans (of tokens, then of pages) per tile, 12.8 us with
// four and one scan of both; the 9 MB that it writes would take 2 of them.
constexpr int kPlanThreads = 1024;
constexpr uint32_t kPlanMost = 1u << 30;   // sums saturate here

__device__ inline uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kPlanMost); }
__device__ inline uint2 sat_add(uint2 a, uint2 b) {
  return uint2{sat_add(a.x, b.x), sat_add(a.y, b.y)};
}

// Exclusive saturating sums over the workgroup's threads of v; *total gets the
// sum.  `part`: LDS, one place per wave.
__device__ inline uint2 block_scan(uint2 v, uint2* part, uint2* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  uint2 x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint2 y = {__shfl_up(x.x, d), __shfl_up(x.y, d)};
    if (lane >= d) x = sat_add(x, y);
  }
  if (lane == 63) part[wave] = x;
  __syncthreads();
  uint2 before = {0, 0}, all = {0, 0};
  for (int w = 0; w < nw; ++w) {
    const uint2 p = part[w];
    if (w < wave) before = sat_add(before, p);
    all = sat_add(all, p);
  }
  const uint2 up = {__shfl_up(x.x, 1), __shfl_up(x.y, 1)};
  __syncthreads();   // `part` may be written again
  *total = all;
  return lane ? sat_add(before, up) : before;
}

struct PlanArgs {
  const int32_t *lengths, *counts, *pool, *taken;
  int32_t *tables, *slots, *positions, *starts, *out_lengths, *out_taken, *status;
  int64_t table_stride;
  int32_t rows, width, pool_size, page_log, capacity, per_block;
  bool wide;   // slots and positions can be written 16 bytes at a time
};

template <int ITEMS>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanArgs a) {
  constexpr int kMost = kPlanThreads * ITEMS;
  __shared__ uint32_t first[kMost + 1], off[kMost];
  __shared__ int32_t len[kMost];
  __shared__ uint2 part[kPlanThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x, tile = nt * ITEMS;
  const uint32_t cap = a.capacity;
  const uint32_t ps = 1u << a.page_log, width = a.width;
  const uint32_t taken = min(max(*a.taken, 0), a.pool_size);
  const uint32_t lo = (uint32_t)blockIdx.x * a.per_block;
  const uint32_t hi = min(lo + (uint32_t)a.per_block, cap);
  uint2 base = {0, 0};   // tokens and pages of the tiles before
  for (int r0 = 0; r0 < a.rows; r0 += tile) {
    uint32_t n[ITEMS], cnt[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int r = r0 + tid * ITEMS + i;
      const bool in = r < a.rows;
      n[i] = in ? (uint32_t)min((int64_t)max(a.lengths[r], 0), (int64_t)width << a.page_log) : 0;
      cnt[i] = in ? min((uint32_t)max(a.counts[r], 0), kPlanMost) : 0;
    }
    const auto pages = [&](int i, uint32_t add) {   // new pages for `add` tokens of row i
      return min((n[i] + add + ps - 1) >> a.page_log, width) - ((n[i] + ps - 1) >> a.page_log);
    };
    uint2 sum = {0, 0}, all;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) sum = sat_add(sum, uint2{cnt[i], pages(i, cnt[i])});
    uint2 at = sat_add(base, block_scan(sum, part, &all));
    if (sat_add(base.x, all.x) > cap) {
      // the slot map ends in this tile: only the tokens before its end take pages
      uint32_t start = at.x;
      sum = uint2{0, 0};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        sum.y += pages(i, start < cap ? min(cnt[i], cap - start) : 0);
        start = sat_add(start, cnt[i]);
      }
      uint2 some;
      at.y = sat_add(base.y, block_scan(sum, part, &some).y);
      all.y = some.y;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int s = tid * ITEMS + i, r = r0 + s;
      const uint32_t add = at.x < cap ? min(cnt[i], cap - at.x) : 0, need = pages(i, add);
      first[s] = at.x;
      off[s] = at.y;
      len[s] = n[i];
      if (blockIdx.x == 0 && r < a.rows) {
        const uint32_t left = a.pool_size - taken;
        const uint32_t got = at.y < left ? min(need, left - at.y) : 0;
        const uint32_t have = (n[i] + ps - 1) >> a.page_log;
        a.starts[r] = at.x;
        a.out_lengths[r] = min(n[i] + add, (have + got) << a.page_log);
        a.status[r] = (got < need ? 1 : 0) |
                      ((n[i] + add + ps - 1) >> a.page_log > width ? 2 : 0) | (add < cnt[i] ? 4 : 0);
        if (r == a.rows - 1) a.starts[a.rows] = sat_add(at.x, cnt[i]);
      }
      at = sat_add(at, uint2{cnt[i], need});
    }
    if (tid == nt - 1) first[tile] = at.x;
    __syncthreads();
    const uint32_t begin = max(lo, base.x), end = min(hi, first[tile]);
    // a thread has four neighbouring tokens: one search, and seldom more than two pages
    for (uint32_t j0 = (begin & ~3u) + 4 * tid; j0 < end; j0 += 4 * nt) {
      // the last row of the tile that starts at or before the first of them (empty rows
      // share a start)
      const uint32_t j1 = max(j0, begin);
      int s = 0;
      for (int step = kMost / 2; step; step >>= 1)
        if (s + step < tile && first[s + step] <= j1) s += step;
      int32_t slot[4], position[4];
      int32_t page = -1;
      uint32_t of = ~0u;   // the page of the row that `page` is
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t j = j0 + i;
        slot[i] = position[i] = -1;
        if (j < begin || j >= end) continue;
        while (j >= first[s + 1]) {
          ++s;
          of = ~0u;
        }
        const uint32_t pos = (uint32_t)len[s] + (j - first[s]), p = pos >> a.page_log;
        if (p != of) {
          const uint32_t held = ((uint32_t)len[s] + ps - 1) >> a.page_log;
          of = p;
          page = -1;
          if (p < width) {
            int32_t* entry = a.tables + (int64_t)(r0 + s) * a.table_stride + p;
            if (p < held) {
              page = *entry;
            } else {
              const uint32_t from = taken + off[s] + (p - held);
              if (from < (uint32_t)a.pool_size) page = a.pool[from];
              if ((pos & (ps - 1)) == 0) *entry = page;
            }
          }
        }
        slot[i] = page < 0 ? -1 : (int32_t)(((uint32_t)page << a.page_log) + (pos & (ps - 1)));
        position[i] = (int32_t)pos;
      }
      if (a.wide && j0 >= begin && j0 + 4 <= end) {
        *reinterpret_cast<int4*>(a.slots + j0) = int4{slot[0], slot[1], slot[2], slot[3]};
        *reinterpret_cast<int4*>(a.positions + j0) =
            int4{position[0], position[1], position[2], position[3]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + i >= begin && j0 + i < end) {
            a.slots[j0 + i] = slot[i];
            a.positions[j0 + i] = position[i];
          }
      }
    }
    base = sat_add(base, all);
    __syncthreads();   // the tile's arrays are rewritten
  }
  for (uint32_t j = max(lo, base.x) + tid; j < hi; j += nt) {
    a.slots[j] = -1;
    a.positions[j] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.out_taken[0] = min(taken + base.y, (uint32_t)a.pool_size);
    if (a.rows == 0) a.starts[0] = 0;
  }
}

struct ReleaseArgs {
  const uint8_t* finished;
  const int32_t *lengths, *tables, *taken;
  int32_t *pool, *out_lengths, *out_taken;
  int64_t table_stride;
  int32_t rows, width, pool_size, page_log;
  int32_t per;   // rows of a workgroup
};

// Two passes: the first counts the pages that come back from all rows (it fixes where
// the first of them goes) and from the rows before the workgroup's own `per`, the second
// moves those of its own rows, a wave per row.  Every workgroup counts for itself, so
// that one launch does: latency again.  4096 rows of 63 pages each: 129 us in one
// workgroup, 8.8 us in 256.
__global__ __launch_bounds__(kPlanThreads) void release_kernel(ReleaseArgs a) {
  __shared__ uint32_t off[kPlanThreads], num[kPlanThreads];
  __shared__ uint2 part[kPlanThreads / 64];
  const int tid = threadIdx.x, nt = blockDim.x;
  const uint32_t ps = 1u << a.page_log;
  const int first = min((int64_t)blockIdx.x * a.per, (int64_t)a.rows);
  const int end = min((int64_t)first + a.per, (int64_t)a.rows);
  const auto pages_of = [&](int r) -> uint32_t {
    if (!a.finished[r]) return 0;
    const uint32_t n =
        (uint32_t)min((int64_t)max(a.lengths[r], 0), (int64_t)a.width << a.page_log);
    return (n + ps - 1) >> a.page_log;
  };
  uint2 mine{0, 0}, sum;   // pages of rows before the workgroup's, and of all
  for (int r = tid; r < a.rows; r += nt) {
    const uint32_t n = pages_of(r);
    mine = sat_add(mine, uint2{r < first ? n : 0, n});
  }
  block_scan(mine, part, &sum);
  const int32_t taken = min(max(*a.taken, 0), a.pool_size);
  const int32_t left = taken - (int32_t)min(sum.y, (uint32_t)taken);
  uint32_t base = sum.x;
  for (int r0 = first; r0 < end; r0 += nt) {
    const int r = r0 + tid;
    const uint32_t n = r < end ? pages_of(r) : 0;
    off[tid] = sat_add(base, block_scan(uint2{0, n}, part, &sum).y);
    num[tid] = n;
    if (r < end) a.out_lengths[r] = a.finished[r] ? 0 : a.lengths[r];
    __syncthreads();
    for (int w = tid >> 6; w < nt && r0 + w < end; w += nt >> 6)
      for (uint32_t k = tid & 63; k < num[w]; k += 64) {
        // a row released twice asks for more pages than were taken: the rest is left out
        const uint32_t at = (uint32_t)left + off[w] + k;
        if (at < (uint32_t)taken) a.pool[at] = a.tables[(int64_t)(r0 + w) * a.table_stride + k];
      }
    base = sat_add(base, sum.y);
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) a.out_taken[0] = left;
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
// looked up once for both.  131072 tokens of 8 x 128 bf16: 200 us, 5.4 TB/s (a copy
// of 2 GiB by the library: 4.9 TB/s).  One token of each of 256 requests: 2.8 us.
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
