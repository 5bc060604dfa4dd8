// Attention of one token per request over a paged key/value cache.
//
// out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = scale q.k_t, in one
// pass over the cache with a running maximum m and sum l: what the kernel
// cannot do without is reading every key and value once, so everything else is
// arranged to keep those loads in flight.
//
// - One workgroup per (request, key/value head, up to 16 of its query heads,
//   part of the length); its four waves take tiles of the part in turn and are
//   joined through LDS, the parts by join_kernel.
// - A wave's tile is 32 tokens (16-bit types) or 16 (f32).  Keys and values go
//   from memory straight into the registers that the matrix instructions read:
//   scores as K (tokens x d) . Q^T (d x heads), the output as V^T (d x tokens) .
//   P^T (tokens x heads).  With the tile's tokens assigned to the rows of the
//   two score products as below, the scores leave the first product in the very
//   lanes in which the second wants them, so nothing crosses lanes but the
//   maximum over four lanes.
// - Lane l = 16 g + c.  Score columns are heads (c).  Row i of score product T
//   is token (i>>2)*8 + T*4 + (i&3), so that lane (g, c) ends up with tokens
//   8g .. 8g+7 of head c: the k-slice of lane group g in the second product.
//   There lane (g, c) holds values of tokens 8g..8g+7 at d = 8c..8c+7 (one
//   16-byte load per token, 256 contiguous bytes per 16 lanes); the transposed
//   operand for d = 8c + j is a byte permutation within the lane.
// - The probabilities of 16-bit types enter the second product as the sum of
//   two values of that type (high part and remainder): the products are not
//   what bounds the kernel, and the output then differs from the exact one by
//   its own rounding only.
#pragma once
#include "cache.h"

namespace ctcpb_lm {

constexpr int kAttnWaves = 4;

struct AttnArgs {
  const char* q;
  char* out;
  float* lse;
  float* part;                    // joined later: [row][head][split][D] then (m, l) pairs
  const int32_t *tables, *lengths;
  int64_t q_r, q_h, out_r, out_h; // strides in elements
  int64_t table_stride;
  CacheView kc, vc;
  int32_t rows, heads, kv_heads, group, head_tiles, D;
  int32_t width, page_log, num_pages, max_len, window;
  int32_t chunk, splits;          // tokens per part, parts per row
  float scale;
};

template <typename T>
struct Elem;

template <>
struct Elem<__bf16> {
  typedef bf16x8 V8;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Elem<_Float16> {
  typedef f16x8 V8;
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Elem<float> {};

// A request's range of tokens [lo, hi), lo rounded down to `tile` in `base`.
struct Range {
  int32_t lo, hi, base;
};
__device__ inline Range attn_range(const AttnArgs& a, int row, int tile) {
  Range r;
  r.hi = min(max(a.lengths[row], 0), a.max_len);
  r.lo = a.window > 0 ? max(r.hi - a.window, 0) : 0;
  r.base = r.lo & ~(tile - 1);
  return r;
}

// State of one wave: for head c of the lane (the same in the four lane groups
// for m; l is this lane group's share).
template <int NA>
struct WaveState {
  float m, l;      // scores stay in natural units: times log2(e), the lowest float is -inf
  f32x4 acc[NA];   // acc[j][r]: see the tile functions for the d each one is
};

// The page of token t's group of four (clamped to the request's last token, so
// that every entry read is one the request owns, and to the cache).
__device__ inline int32_t group_page(const AttnArgs& a, const int32_t* table, int32_t t,
                                     int32_t last) {
  const int32_t p = table[min(t, last) >> a.page_log];
  return min((uint32_t)p, (uint32_t)(a.num_pages - 1));
}

// ---- 16-bit types: 32 tokens x DP (64, 128 or 256) -----------------------
template <typename T, int DP>
struct Tile {
  static constexpr int kTokens = 32;
  static constexpr int kK = DP / 32;            // k-steps of the score product
  static constexpr int kV = DP >= 128 ? 8 : 4;  // values a lane loads at once
  static constexpr int kH = DP / 16 / kV;       // such loads per token
  static constexpr int kAcc = DP / 16;
  typedef typename Elem<T>::V8 V8;
  typedef V8 Query[kK];

  static __device__ void load_query(const AttnArgs& a, const T* q, bool live, Query& f) {
    const int g = (threadIdx.x & 63) >> 4;
    for (int k = 0; k < kK; ++k)
      for (int i = 0; i < 8; ++i) {
        const int d = k * 32 + g * 8 + i;
        f[k][i] = live && d < a.D ? q[d] : (T)0.0f;
      }
  }

  // d of acc[j][r] in this lane
  static __device__ int dim_of(int j, int r) {
    const int g = (threadIdx.x & 63) >> 4;
    return (j / kV) * (16 * kV) + (g * 4 + r) * kV + j % kV;
  }

  static __device__ void step(const AttnArgs& a, const char* kbase, const char* vbase,
                              const int32_t* table, int32_t t0, const Range& rg, const Query& q,
                              float scale, WaveState<kAcc>& s) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    // the pages of the tile's eight groups of four tokens, one per lane 0..7
    const int32_t pg = group_page(a, table, t0 + (lane & 7) * 4, rg.hi - 1);
    V8 kf[2][kK];
    for (int h = 0; h < 2; ++h) {
      const int grp = (c >> 2) * 2 + h;
      const int64_t page = __shfl(pg, grp);
      const int32_t t = t0 + grp * 4 + (c & 3);
      const char* p = kbase + page * a.kc.page + (int64_t)(t & mask) * a.kc.token;
      for (int k = 0; k < kK; ++k) {
        const int d = k * 32 + g * 8;
        u32x4 z = {0, 0, 0, 0};
        if (d < a.D) z = *reinterpret_cast<const u32x4*>(p + d * 2);
        kf[h][k] = __builtin_bit_cast(V8, z);
      }
    }
    uint32_t vr[8][kH][kV / 2];
    for (int h = 0; h < 2; ++h) {
      const int grp = g * 2 + h;
      const int64_t page = __shfl(pg, grp);
      for (int i = 0; i < 4; ++i) {
        const int32_t t = t0 + grp * 4 + i;
        const char* p = vbase + page * a.vc.page + (int64_t)(t & mask) * a.vc.token;
        for (int b = 0; b < kH; ++b) {
          const int d = b * 16 * kV + c * kV;
          if constexpr (kV == 8) {
            u32x4 z = {0, 0, 0, 0};
            if (d < a.D) z = *reinterpret_cast<const u32x4*>(p + d * 2);
            for (int x = 0; x < 4; ++x) vr[h * 4 + i][b][x] = z[x];
          } else {
            u32x2 z = {0, 0};
            if (d < a.D) z = *reinterpret_cast<const u32x2*>(p + d * 2);
            for (int x = 0; x < 2; ++x) vr[h * 4 + i][b][x] = z[x];
          }
        }
      }
    }
    f32x4 sc[2] = {};
    for (int h = 0; h < 2; ++h)
      for (int k = 0; k < kK; ++k) sc[h] = Elem<T>::mfma(kf[h][k], q[k], sc[h]);
    const bool whole = t0 >= rg.lo && t0 + 32 <= rg.hi;
    float p[8];
    float top = neg_inf();
    for (int i = 0; i < 8; ++i) {
      p[i] = sc[i >> 2][i & 3] * scale;
      if (!whole) {
        const int32_t t = t0 + g * 8 + i;
        if (t < rg.lo || t >= rg.hi) {
          p[i] = neg_inf();
          // a masked slot may hold anything, and 0 * NaN is NaN
          for (int b = 0; b < kH; ++b)
            for (int x = 0; x < kV / 2; ++x) vr[i][b][x] = 0;
        }
      }
      top = fmaxf(top, p[i]);
    }
    const float m = fmaxf(s.m, max_over_groups(top));
    const float m0 = m == neg_inf() ? 0.0f : m;   // nothing seen yet: avoid inf - inf
    const float alpha = exp_fast(s.m - m0);
    s.m = m;
    s.l *= alpha;
    V8 hi, lo;
    for (int i = 0; i < 8; ++i) {
      p[i] = exp_fast(p[i] - m0);
      s.l += p[i];
      hi[i] = (T)p[i];
      lo[i] = (T)(p[i] - (float)hi[i]);
    }
    for (int b = 0; b < kH; ++b)
      for (int j = 0; j < kV; ++j) {
        u32x4 w;
        for (int i = 0; i < 4; ++i)
          w[i] = __builtin_amdgcn_perm(vr[2 * i + 1][b][j / 2], vr[2 * i][b][j / 2],
                                       j & 1 ? 0x07060302u : 0x05040100u);
        const V8 vf = __builtin_bit_cast(V8, w);
        f32x4 o = s.acc[b * kV + j] * alpha;
        o = Elem<T>::mfma(vf, hi, o);
        s.acc[b * kV + j] = Elem<T>::mfma(vf, lo, o);
      }
  }
};

// ---- f32: 16 tokens x DP -------------------------------------------------
template <int DP>
struct Tile<float, DP> {
  static constexpr int kTokens = 16;
  static constexpr int kK = DP / 16;
  static constexpr int kH = DP / 64;
  static constexpr int kAcc = DP / 16;
  typedef f32x4 Query[kK];

  static __device__ void load_query(const AttnArgs& a, const float* q, bool live, Query& f) {
    const int g = (threadIdx.x & 63) >> 4;
    for (int k = 0; k < kK; ++k)
      for (int i = 0; i < 4; ++i) {
        const int d = k * 16 + g * 4 + i;
        f[k][i] = live && d < a.D ? q[d] : 0.0f;
      }
  }

  static __device__ int dim_of(int j, int r) {
    const int g = (threadIdx.x & 63) >> 4;
    return (j / 4) * 64 + (g * 4 + r) * 4 + j % 4;
  }

  static __device__ void step(const AttnArgs& a, const char* kbase, const char* vbase,
                              const int32_t* table, int32_t t0, const Range& rg, const Query& q,
                              float scale, WaveState<kAcc>& s) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    const int32_t pg = group_page(a, table, t0 + (lane & 3) * 4, rg.hi - 1);
    f32x4 kf[kK];
    {
      const int64_t page = __shfl(pg, c >> 2);
      const char* p = kbase + page * a.kc.page + (int64_t)((t0 + c) & mask) * a.kc.token;
      for (int k = 0; k < kK; ++k) {
        const int d = k * 16 + g * 4;
        kf[k] = f32x4{0, 0, 0, 0};
        if (d < a.D) kf[k] = *reinterpret_cast<const f32x4*>(p + d * 4);
      }
    }
    f32x4 vf[4][kH];
    {
      const int64_t page = __shfl(pg, g);
      for (int r = 0; r < 4; ++r) {
        const char* p =
            vbase + page * a.vc.page + (int64_t)((t0 + g * 4 + r) & mask) * a.vc.token;
        for (int b = 0; b < kH; ++b) {
          const int d = b * 64 + c * 4;
          vf[r][b] = f32x4{0, 0, 0, 0};
          if (d < a.D) vf[r][b] = *reinterpret_cast<const f32x4*>(p + d * 4);
        }
      }
    }
    f32x4 sc = {};
    for (int k = 0; k < kK; ++k)
      for (int i = 0; i < 4; ++i)
        sc = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[k][i], q[k][i], sc, 0, 0, 0);
    const bool whole = t0 >= rg.lo && t0 + 16 <= rg.hi;
    float top = neg_inf();
    for (int r = 0; r < 4; ++r) {
      sc[r] *= scale;
      if (!whole) {
        const int32_t t = t0 + g * 4 + r;
        if (t < rg.lo || t >= rg.hi) {
          sc[r] = neg_inf();
          for (int b = 0; b < kH; ++b) vf[r][b] = f32x4{0, 0, 0, 0};
        }
      }
      top = fmaxf(top, sc[r]);
    }
    const float m = fmaxf(s.m, max_over_groups(top));
    const float m0 = m == neg_inf() ? 0.0f : m;
    const float alpha = exp_of<float>(s.m - m0);
    s.m = m;
    s.l *= alpha;
    for (int r = 0; r < 4; ++r) {
      sc[r] = exp_of<float>(sc[r] - m0);
      s.l += sc[r];
    }
    for (int b = 0; b < kH; ++b)
      for (int i = 0; i < 4; ++i) {
        f32x4 o = s.acc[b * 4 + i] * alpha;
        for (int r = 0; r < 4; ++r)
          o = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[r][b][i], sc[r], o, 0, 0, 0);
        s.acc[b * 4 + i] = o;
      }
  }
};

template <typename T, int DP>
__global__ __launch_bounds__(64 * kAttnWaves) void attn_kernel(AttnArgs a) {
  typedef Tile<T, DP> TL;
  __shared__ float acc[kAttnWaves][16][DP + 4];
  __shared__ float ms[kAttnWaves][16], ls[kAttnWaves][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  int64_t id = blockIdx.x;
  const int split = (int)(id % a.splits);
  id /= a.splits;
  const int ht = (int)(id % a.head_tiles);
  id /= a.head_tiles;
  const int kvh = (int)(id % a.kv_heads), row = (int)(id / a.kv_heads);
  const Range rg = attn_range(a, row, TL::kTokens);
  const int32_t begin = rg.base + split * a.chunk;
  const int32_t end = min(rg.hi, begin + a.chunk);
  if (a.splits > 1 && begin >= end) return;   // join_kernel does not look at it either
  const int nh = min(16, a.group - ht * 16);  // query heads of this block
  const int head0 = kvh * a.group + ht * 16;
  const bool live = c < nh;
  typename TL::Query q;
  TL::load_query(a, reinterpret_cast<const T*>(a.q) + row * a.q_r + (head0 + (live ? c : 0)) * a.q_h,
                 live, q);
  WaveState<TL::kAcc> s;
  s.m = neg_inf();
  s.l = 0.0f;
  for (int j = 0; j < TL::kAcc; ++j) s.acc[j] = f32x4{0, 0, 0, 0};
  const int32_t* table = a.tables + row * a.table_stride;
  const char* kbase = a.kc.data + kvh * a.kc.head;
  const char* vbase = a.vc.data + kvh * a.vc.head;
  for (int32_t t = begin + wave * TL::kTokens; t < end; t += kAttnWaves * TL::kTokens)
    TL::step(a, kbase, vbase, table, t, rg, q, a.scale, s);
  // join the waves
  const float l = sum_over_groups(s.l);
  if (g == 0) {
    ms[wave][c] = s.m;
    ls[wave][c] = l;
  }
  for (int j = 0; j < TL::kAcc; ++j)
    for (int r = 0; r < 4; ++r) acc[wave][c][TL::dim_of(j, r)] = s.acc[j][r];
  __syncthreads();
  for (int i = threadIdx.x; i < nh * a.D; i += 64 * kAttnWaves) {
    const int h = i / a.D, d = i % a.D;
    float m = neg_inf();
    for (int w = 0; w < kAttnWaves; ++w) m = fmaxf(m, ms[w][h]);
    const float m0 = m == neg_inf() ? 0.0f : m;
    float sum = 0.0f, o = 0.0f;
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = exp_of<T>(ms[w][h] - m0);
      sum += f * ls[w][h];
      o += f * acc[w][h][d];
    }
    const int64_t rh = (int64_t)row * a.heads + head0 + h;
    if (a.splits == 1) {
      reinterpret_cast<T*>(a.out)[row * a.out_r + (head0 + h) * a.out_h + d] =
          (T)(sum == 0.0f ? 0.0f : o / sum);
      if (d == 0 && a.lse) a.lse[rh] = sum == 0.0f ? neg_inf() : m + __log2f(sum) * kLn2;
    } else {
      a.part[(rh * a.splits + split) * a.D + d] = o;
      if (d == 0) {
        float* ml = a.part + (int64_t)a.rows * a.heads * a.splits * a.D;
        ml[2 * (rh * a.splits + split)] = m;
        ml[2 * (rh * a.splits + split) + 1] = sum;
      }
    }
  }
}

// Joins the parts of one (request, head), in their order.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, int tile) {
  const int64_t rh = blockIdx.x;
  const int row = (int)(rh / a.heads), head = (int)(rh % a.heads);
  const Range rg = attn_range(a, row, tile);
  const int n = rg.hi > rg.base ? (rg.hi - rg.base + a.chunk - 1) / a.chunk : 0;
  const float* ml = a.part + (int64_t)a.rows * a.heads * a.splits * a.D + 2 * rh * a.splits;
  float m = neg_inf();
  for (int s = 0; s < n; ++s) m = fmaxf(m, ml[2 * s]);
  const float m0 = m == neg_inf() ? 0.0f : m;
  const int d = threadIdx.x;
  float sum = 0.0f, o = 0.0f;
  for (int s = 0; s < n; ++s) {
    const float f = exp_of<T>(ml[2 * s] - m0);
    sum += f * ml[2 * s + 1];
    if (d < a.D) o += f * a.part[(rh * a.splits + s) * a.D + d];
  }
  if (d < a.D)
    reinterpret_cast<T*>(a.out)[row * a.out_r + head * a.out_h + d] =
        (T)(sum == 0.0f ? 0.0f : o / sum);
  if (d == 0 && a.lse) a.lse[rh] = sum == 0.0f ? neg_inf() : m + __log2f(sum) * kLn2;
}

}  // namespace ctcpb_lm
