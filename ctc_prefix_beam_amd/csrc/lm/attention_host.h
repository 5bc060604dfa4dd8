// The launches of an attention call.
#pragma once
#include <algorithm>

#include "attention.h"
#include "host.h"

namespace ctcpb_lm {

// The launch plan of an attention call, a function of sizes only (the lengths
// stay on the device).
struct AttnPlan {
  int32_t head_tiles, max_len, waves, ranges;
  int64_t items;
  size_t o_part, bytes;   // workspace: the rows' prefix sums, then the parts
};

inline int32_t length_bound(const ctcpb_lm_attention_args& g) {
  const int32_t held = g.table_width * g.page_size;
  return g.max_len == 0 || g.max_len > held ? held : g.max_len;
}

inline int check_attention(const ctcpb_lm_attention_args& g) {
  if (!elem_size(g.dtype)) return fail(CTCPB_ERR_INVALID, kBadType);
  if (g.kv_heads < 1 || g.q_heads < g.kv_heads || g.q_heads % g.kv_heads)
    return fail(CTCPB_ERR_INVALID, "q_heads must be a multiple of kv_heads >= 1");
  if (g.head_dim < 8 || g.head_dim % 8)
    return fail(CTCPB_ERR_INVALID, "head_dim must be a multiple of 8");
  if (g.head_dim > 256) return fail(CTCPB_ERR_UNSUPPORTED, "head_dim above 256");
  if (g.max_len < 0 || g.window < 0)
    return fail(CTCPB_ERR_INVALID, "max_len and window must be >= 0");
  return check_table(g.rows, g.table_stride, g.table_width, g.page_size);
}

// The kernels' arguments of a call that check_attention() has passed, with the rest of its
// checks; nothing of `a` counts where there are no rows.  cache_es: bytes of a value in the
// caches; `small`: the error of too small a workspace.
inline int attention_args(const ctcpb_lm_attention_args& g, const AttnPlan& p, int cache_es,
                          void* workspace, size_t workspace_bytes, const char* small,
                          AttnArgs& a) {
  const int es = elem_size(g.dtype);
  if (int rc = check_pages(g.num_pages, g.page_size)) return rc;
  if (g.q_stride_r < 0 || g.q_stride_h < 0 || g.out_stride_r < 0 || g.out_stride_h < 0)
    return fail(CTCPB_ERR_INVALID, "strides must be >= 0");
  if (int rc = check_cache(g.k_cache)) return rc;
  if (int rc = check_cache(g.v_cache)) return rc;
  a.kc = view(g.k_cache, cache_es);
  a.vc = view(g.v_cache, cache_es);
  if (!wide_cache(a.kc) || !wide_cache(a.vc))
    return fail(CTCPB_ERR_INVALID,
                "caches must be 16-byte aligned, with strides that are multiples of 16 bytes");
  if (g.rows == 0) return CTCPB_OK;
  if (!g.q || !g.out || !g.lengths || (!g.tables && g.table_width))
    return fail(CTCPB_ERR_INVALID, kNull);
  if (p.bytes && (!workspace || !aligned(workspace, 16)))
    return fail(CTCPB_ERR_INVALID, "workspace must be 16-byte aligned and not NULL");
  if (workspace_bytes < p.bytes)
    return fail(CTCPB_ERR_TOO_SMALL, small);
  // steps of all rows are counted with 31 bits
  if (p.items > INT_MAX || (int64_t)g.rows * g.q_heads > INT_MAX ||
      (int64_t)g.rows * (p.max_len / 64 + 1) > INT_MAX)
    return fail(CTCPB_ERR_UNSUPPORTED, "too many rows for one launch");
  a.q = static_cast<const char*>(g.q);
  a.out = static_cast<char*>(g.out);
  a.lse = g.lse;
  a.prefix = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.o_part);
  a.tables = g.tables;
  a.lengths = g.lengths;
  a.q_r = g.q_stride_r;
  a.q_h = g.q_stride_h;
  a.out_r = g.out_stride_r;
  a.out_h = g.out_stride_h;
  a.table_stride = g.table_stride;
  a.rows = g.rows;
  a.heads = g.q_heads;
  a.kv_heads = g.kv_heads;
  a.group = g.q_heads / g.kv_heads;
  a.head_tiles = p.head_tiles;
  a.D = g.head_dim;
  a.width = g.table_width;
  a.page_log = log2_of(g.page_size);
  a.num_pages = g.num_pages;
  a.max_len = p.max_len;
  a.window = g.window;
  a.items = (int32_t)p.items;
  a.ranges = p.ranges;
  a.wide_q = aligned(g.q, 16) && g.q_stride_r * es % 16 == 0 && g.q_stride_h * es % 16 == 0;
  a.wide_out =
      aligned(g.out, 16) && g.out_stride_r * es % 16 == 0 && g.out_stride_h * es % 16 == 0;
  a.scale = g.scale;
  return CTCPB_OK;
}

// A CU's LDS, of which kernels that are given theirs at the launch have none of their own.
constexpr int kLds = 160 * 1024;

// Whether `kernel` was launched; if not, the error is the thread's last one.  How much LDS a kernel
// may be given is noted for the kernel, not for the call: always the same, so that calls of
// several threads do not take it from each other.
template <typename K, typename Args>
bool launch_with_lds(K kernel, unsigned blocks, int threads, size_t lds, const Args& a,
                     hipStream_t st) {
  if (lds > 65536 &&   // more than a kernel has unasked
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, kLds) != hipSuccess)
    return false;
  kernel<<<blocks, threads, lds, st>>>(a);
  return true;
}

template <typename TL>
void launch_tiles_of(const typename TL::Args& a, const AttnPlan& p, hipStream_t st) {
  const size_t state = (size_t)std::min(16, a.group) * (TL::kDP + 6) * sizeof(float);
  if (p.waves == 1) {
    attn_kernel<TL, 1><<<(unsigned)((p.items + 3) / 4), 256, 0, st>>>(a);
  } else if (p.waves) {
    constexpr int NW = TL::kDP <= 128 ? 8 : 4;
    launch_with_lds(attn_kernel<TL, NW>, (unsigned)p.items, 64 * NW, NW * state, a, st);
  } else {
    const bool done = launch_with_lds(
        attn_range_kernel<TL>, (unsigned)((int64_t)p.ranges * a.kv_heads * a.head_tiles),
        64 * kRangeWaves, kRangeWaves * state, a, st);
    if (!done || p.ranges == 1) return;   // (one range: no row is split)
    constexpr int kGroups = 256 / (TL::kDP / 4);
    const int64_t heads = (int64_t)a.rows * a.heads;
    // a workgroup to each head while that does not make more than a few to a CU
    const int ways = heads <= 1024 ? kGroups : 1, per = kGroups / ways;
    join_kernel<TL><<<(unsigned)((heads + per - 1) / per), 256, 0, st>>>(a, ways);
  }
}

}  // namespace ctcpb_lm
