// Attention of one token per request over a paged key/value cache.
//
// out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = scale q.k_t, in one
// pass over the cache with a running maximum m and sum l: what the kernel
// cannot do without is reading every key and value once, so everything else is
// arranged to keep those loads in flight.
//
// - Short requests: eight waves share a request's tiles for one key/value head
//   (and up to 16 of its query heads).  Very many of them: a wave has a request
//   and head for itself, and the four waves of a workgroup take neighbouring heads
//   of the same tokens.  Both are one launch.
// - Otherwise the tokens of all requests, laid end to end, are cut into ranges of
//   equal length, as many as workgroups fit on the card, whatever the requests'
//   own lengths (the kernel finds its range from the prefix sums of the lengths);
//   four waves take a range's tiles in turn.  A request that lies in several
//   ranges leaves a part in each, joined in their order by join_kernel.
// - A wave's registers hold one tile of keys and one of values; the next keys are
//   fetched when the scores are done, the next values when the output is, so some
//   loads are always under way.
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
//   two values of that type (high part and remainder), which have 16 bits together
//   (bf16) or 22: the products are not what bounds the kernel, and the output then
//   differs from the exact one by its own rounding and some 2^-17 of the values.  f16
//   ends at 2^-24, so its probabilities are multiplied by 2^15 first: without that, what
//   a wave added for tokens 17 below the largest score it had met was 1.4 times too
//   much, and nothing for those 18 below, while the sum l counted them in full.
//
// What bounds it, measured: memory.  256 requests of 1..4095 tokens, 32 query and 8
// key/value heads of 128, bf16: 2.15 GB in 419 us, 5.1 TB/s, where a kernel that only
// reads so much gets 6.3 to 6.5 TB/s from one long run of addresses and 435 / 411 us
// from pages laid token by token / head by head; three requests of up to 131071
// tokens, head by head: 1.21 GB in 229 us, 5.3 TB/s; 4096 requests of up to 512
// tokens, 4 heads of 64, f16: 1.08 GB in 219 us, 4.9 TB/s.  One request of a few
// hundred tokens: 12 us, the latency of a handful of dependent loads (lengths, table,
// keys, values) and the join of eight waves.
#pragma once
#include "common.h"

namespace ctcpb_lm {

// Ranges are counted in steps of the four waves' tiles, at least kLeastSteps each: with
// shorter ones, joining costs what splitting gains.  One request of 30000 tokens takes
// 36 us with 4, 30 with 8; 32 requests of 100 to 2000 tokens 38 us with 4, 40 with 8.
// Where the rows' average is less, it is that: shorter rows are then not done one after
// another by a few workgroups (64 requests of up to 64 tokens, with tables of 8192: 19.9 us
// with six always, 9.5 so).
constexpr int kRangeWaves = 4;
constexpr int kLeastSteps = 6;

struct AttnArgs {
  const char* q;
  char* out;
  float* lse;
  int32_t* prefix;                // ranges: [rows + 1] steps of the rows before
  float* part;                    // ranges: parts of split rows, D values, m and l each
  const int32_t *tables, *lengths;
  int64_t q_r, q_h, out_r, out_h; // strides in elements
  int64_t table_stride;
  CacheView kc, vc;
  int32_t rows, heads, kv_heads, group, head_tiles, D;
  int32_t width, page_log, num_pages, max_len, window;
  int32_t items;                  // (row, key/value head, head tile)
  int32_t ranges;                 // of the tokens, for each key/value head and head tile
  bool wide_q, wide_out;          // rows of q / out can be accessed 16 bytes at a time
  float scale;
};

template <typename T>
struct Elem;

template <>
struct Elem<__bf16> {
  typedef bf16x8 V8;
  static constexpr float kRaise = 1.0f;   // of the probabilities in the second product
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Elem<_Float16> {
  typedef f16x8 V8;
  static constexpr float kRaise = 32768.0f;   // the largest power of two that f16 holds
  static __device__ f32x4 mfma(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Elem<float> {
  static constexpr float kRaise = 1.0f;
};

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

// The same for a row that is the same in all lanes, kept in scalar registers.
__device__ inline Range attn_range_uniform(const AttnArgs& a, int row, int tile) {
  Range r = attn_range(a, row, tile);
  r.lo = __builtin_amdgcn_readfirstlane(r.lo);
  r.hi = __builtin_amdgcn_readfirstlane(r.hi);
  r.base = __builtin_amdgcn_readfirstlane(r.base);
  return r;
}

// State of one wave: for head c of the lane (the same in the four lane groups
// for m; l is this lane group's share).
template <int NA>
struct WaveState {
  float m, l;      // scores stay in natural units: times log2(e), the lowest float is -inf
  f32x4 acc[NA];   // kRaise times the sums; acc[j][r]: see the tile functions for the d

  __device__ void reset() {
    m = neg_inf();
    l = 0.0f;
#pragma unroll
    for (int j = 0; j < NA; ++j) acc[j] = f32x4{0, 0, 0, 0};
  }
};

// The page of token t's group of four.  It does not wait for the request's length:
// past the last token the entry may be any (kept inside the table and the cache),
// for the tokens there are masked whatever the page holds.
__device__ inline int32_t group_page(const AttnArgs& a, const int32_t* table, int32_t t) {
  const int32_t p = table[min(t >> a.page_log, a.width - 1)];
  return min((uint32_t)p, (uint32_t)(a.num_pages - 1));
}

// Where a wave's tile lies: its first token, and the page of the lane's group of
// four tokens (lane & 7 for 16-bit types, lane & 3 for f32).
struct Spot {
  int32_t t0, page;
};

// ---- 16-bit types: 32 tokens x DP (64, 128 or 256) -----------------------
template <typename T, int DP>
struct Tile {
  typedef T Type;
  typedef AttnArgs Args;
  static constexpr int kDP = DP;
  static constexpr int kAloneWaves = DP == 64 ? 4 : 1;   // on a SIMD: a wave to an item
  static constexpr int kRangeOnSimd = DP == 64 ? 4 : DP == 128 ? 3 : 1;   // and ranges
  static constexpr int kTokens = 32;
  static constexpr bool kWalks = false;   // has a loop over tiles of its own
  static constexpr bool kLimit = false;   // values may be past the type's largest
  static constexpr int kK = DP / 32;            // k-steps of the score product
  static constexpr int kV = DP >= 128 ? 8 : 4;  // values a lane loads at once
  static constexpr int kH = DP / 16 / kV;       // such loads per token
  static constexpr int kAcc = DP / 16;
  typedef typename Elem<T>::V8 V8;
  typedef WaveState<kAcc> State;

  // what takes the sums' factor away
  static __device__ float lower(const State&) { return 1.0f / Elem<T>::kRaise; }
  // neighbouring items that are done on the same XCD
  static __device__ int together(const Args& a) { return a.head_tiles; }

  __device__ void head(const Args&, int) {}

  V8 q[kK], kf[2][kK];
  uint32_t vr[8][kH][kV / 2];

  __device__ void load_query(const AttnArgs& a, const T* src, bool live) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int d = k * 32 + g * 8;
      u32x4 z = {0, 0, 0, 0};
      if (live && d < a.D) {
        if (a.wide_q) {
          z = *reinterpret_cast<const u32x4*>(src + d);
        } else {
          V8 f;
          for (int i = 0; i < 8; ++i) f[i] = src[d + i];
          z = __builtin_bit_cast(u32x4, f);
        }
      }
      q[k] = __builtin_bit_cast(V8, z);
    }
  }

  // acc[j][r] is d = run_of(r) + j for the kV values j of a load; loads are 16 kV apart
  static constexpr int kRun = kV;
  static __device__ int run_of(int b, int r) {
    return b * 16 * kV + (((threadIdx.x & 63) >> 4) * 4 + r) * kV;
  }

  static __device__ Spot spot(const AttnArgs& a, const int32_t* table, int32_t t0, int) {
    return Spot{t0, group_page(a, table, t0 + (threadIdx.x & 7) * 4)};
  }

  __device__ void load_keys(const AttnArgs& a, const char* base, const Spot& at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int grp = (c >> 2) * 2 + h;
      const int64_t page = __shfl(at.page, grp);
      const int32_t t = at.t0 + grp * 4 + (c & 3);
      const char* p = base + page * a.kc.page + (int64_t)(t & mask) * a.kc.token;
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int d = k * 32 + g * 8;
        u32x4 z = {0, 0, 0, 0};
        if (d < a.D) z = *reinterpret_cast<const u32x4*>(p + d * 2);
        kf[h][k] = __builtin_bit_cast(V8, z);
      }
    }
  }

  __device__ void load_values(const AttnArgs& a, const char* base, const Spot& at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int grp = g * 2 + h;
      const int64_t page = __shfl(at.page, grp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t t = at.t0 + grp * 4 + i;
        const char* p = base + page * a.vc.page + (int64_t)(t & mask) * a.vc.token;
#pragma unroll
        for (int b = 0; b < kH; ++b) {
          const int d = b * 16 * kV + c * kV;
          if constexpr (kV == 8) {
            u32x4 z = {0, 0, 0, 0};
            if (d < a.D) z = *reinterpret_cast<const u32x4*>(p + d * 2);
#pragma unroll
            for (int x = 0; x < 4; ++x) vr[h * 4 + i][b][x] = z[x];
          } else {
            u32x2 z = {0, 0};
            if (d < a.D) z = *reinterpret_cast<const u32x2*>(p + d * 2);
#pragma unroll
            for (int x = 0; x < 2; ++x) vr[h * 4 + i][b][x] = z[x];
          }
        }
      }
    }
  }

  // Scores of the lane's eight tokens t0 + 8g .. for head c.
  __device__ void scores(f32x4 (&sc)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[h] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kK; ++k) sc[h] = Elem<T>::mfma(kf[h][k], q[k], sc[h]);
    }
  }

  __device__ void add(const AttnArgs& a, int32_t t0, const Range& rg, const f32x4 (&sc)[2],
                      WaveState<kAcc>& s) {
    const int g = (threadIdx.x & 63) >> 4;
    const bool whole = t0 >= rg.lo && t0 + 32 <= rg.hi;
    float p[8];
    float top = neg_inf();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = sc[i >> 2][i & 3] * a.scale;
      if (!whole) {
        const int32_t t = t0 + g * 8 + i;
        if (t < rg.lo || t >= rg.hi) {
          p[i] = neg_inf();
          // a masked slot may hold anything, and 0 * NaN is NaN
#pragma unroll
          for (int b = 0; b < kH; ++b)
#pragma unroll
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp_fast(p[i] - m0);
      s.l += p[i];
      const float x = p[i] * Elem<T>::kRaise;
      hi[i] = (T)x;
      lo[i] = (T)(x - (float)hi[i]);
    }
#pragma unroll
    for (int b = 0; b < kH; ++b)
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        u32x4 w;
#pragma unroll
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
  typedef float Type;
  typedef AttnArgs Args;
  static constexpr int kDP = DP;
  static constexpr int kAloneWaves = DP == 64 ? 4 : 1;
  static constexpr int kRangeOnSimd = DP == 64 ? 4 : 1;
  static constexpr int kTokens = 16;
  static constexpr bool kWalks = false;
  static constexpr bool kLimit = false;
  static constexpr int kK = DP / 16;
  static constexpr int kH = DP / 64;
  static constexpr int kAcc = DP / 16;

  typedef WaveState<kAcc> State;

  // what takes the sums' factor away
  static __device__ float lower(const State&) { return 1.0f / Elem<float>::kRaise; }
  // neighbouring items that are done on the same XCD
  static __device__ int together(const Args& a) { return a.head_tiles; }

  __device__ void head(const Args&, int) {}

  f32x4 q[kK], kf[kK], vf[4][kH];

  __device__ void load_query(const AttnArgs& a, const float* src, bool live) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int d = k * 16 + g * 4;
      q[k] = f32x4{0, 0, 0, 0};
      if (live && d < a.D) {
        if (a.wide_q)
          q[k] = *reinterpret_cast<const f32x4*>(src + d);
        else
          for (int i = 0; i < 4; ++i) q[k][i] = src[d + i];
      }
    }
  }

  static constexpr int kRun = 4;
  static __device__ int run_of(int b, int r) {
    return b * 64 + (((threadIdx.x & 63) >> 4) * 4 + r) * 4;
  }

  static __device__ Spot spot(const AttnArgs& a, const int32_t* table, int32_t t0, int) {
    return Spot{t0, group_page(a, table, t0 + (threadIdx.x & 3) * 4)};
  }

  __device__ void load_keys(const AttnArgs& a, const char* base, const Spot& at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    const int64_t page = __shfl(at.page, c >> 2);
    const char* p = base + page * a.kc.page + (int64_t)((at.t0 + c) & mask) * a.kc.token;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int d = k * 16 + g * 4;
      kf[k] = f32x4{0, 0, 0, 0};
      if (d < a.D) kf[k] = *reinterpret_cast<const f32x4*>(p + d * 4);
    }
  }

  __device__ void load_values(const AttnArgs& a, const char* base, const Spot& at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    const int64_t page = __shfl(at.page, g);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const char* p = base + page * a.vc.page + (int64_t)((at.t0 + g * 4 + r) & mask) * a.vc.token;
#pragma unroll
      for (int b = 0; b < kH; ++b) {
        const int d = b * 64 + c * 4;
        vf[r][b] = f32x4{0, 0, 0, 0};
        if (d < a.D) vf[r][b] = *reinterpret_cast<const f32x4*>(p + d * 4);
      }
    }
  }

  // Scores of the lane's four tokens t0 + 4g .. for head c (sc[1] is not used).
  __device__ void scores(f32x4 (&sc)[2]) const {
    sc[0] = sc[1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sc[i & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[k][i], q[k][i], sc[i & 1], 0, 0, 0);
    sc[0] += sc[1];
  }

  __device__ void add(const AttnArgs& a, int32_t t0, const Range& rg, const f32x4 (&sc)[2],
                      WaveState<kAcc>& s) {
    const int g = (threadIdx.x & 63) >> 4;
    const bool whole = t0 >= rg.lo && t0 + 16 <= rg.hi;
    f32x4 p = sc[0] * a.scale;
    float top = neg_inf();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (!whole) {
        const int32_t t = t0 + g * 4 + r;
        if (t < rg.lo || t >= rg.hi) {
          p[r] = neg_inf();
#pragma unroll
          for (int b = 0; b < kH; ++b) vf[r][b] = f32x4{0, 0, 0, 0};
        }
      }
      top = fmaxf(top, p[r]);
    }
    const float m = fmaxf(s.m, max_over_groups(top));
    const float m0 = m == neg_inf() ? 0.0f : m;
    const float alpha = exp_of<float>(s.m - m0);
    s.m = m;
    s.l *= alpha;
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r] = exp_of<float>(p[r] - m0);
    s.l += (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
    for (int b = 0; b < kH; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the tile's sum by itself, then onto the rest: shorter chains of roundings
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          o = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[r][b][i], p[r], o, 0, 0, 0);
        s.acc[b * 4 + i] = s.acc[b * 4 + i] * alpha + o;
      }
  }
};

// Stores N neighbouring values of a head's output, rounded.  LIMIT: a finite one past f16's largest
// becomes that.
template <typename T, int N, bool LIMIT>
__device__ inline void store_run(const AttnArgs& a, int row, int head, int d, const float (&v)[N]) {
  if (d >= a.D) return;
  T* to = reinterpret_cast<T*>(a.out) + row * a.out_r + head * a.out_h + d;
  constexpr int M = N * (int)sizeof(T) <= 16 ? N : 16 / (int)sizeof(T);   // 16 bytes at most
  typedef T TM __attribute__((ext_vector_type(M)));
#pragma unroll
  for (int x = 0; x < N; x += M) {
    TM t;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      float y = v[x + i];
      if (LIMIT && fabsf(y) < __builtin_huge_valf()) y = fminf(fmaxf(y, -65504.0f), 65504.0f);
      t[i] = (T)y;
    }
    if (a.wide_out) {
      *reinterpret_cast<TM*>(to + x) = t;
    } else {
#pragma unroll
      for (int i = 0; i < M; ++i) to[x + i] = t[i];
    }
  }
}

// The hardware's logarithm: over drawn cases lse is 0.57 (bf16), 0.64 (f16) and 1.02 (f32)
// times 2^-24 (1 + |lse|) off at the root mean square, with the library's 0.60, 0.67 and
// 1.04, also where the tiles' exponentials are the library's too.
__device__ inline void store_lse(const AttnArgs& a, int row, int head, float m, float l) {
  if (a.lse)
    a.lse[(int64_t)row * a.heads + head] = l == 0.0f ? neg_inf() : m + __log2f(l) * kLn2;
}

// What the waves of a workgroup do for one head tile of one key/value head.
template <typename TL>
struct Attend {
  typedef typename TL::Type T;
  typedef typename TL::Args Args;
  static constexpr int DP = TL::kDP;
  static constexpr int kRun = TL::kRun, kRuns = TL::kAcc / kRun;
  static constexpr int kPitch = DP + 4;   // a head's place in LDS, and in `part` D + 2

  int head0, nh;
  const char *kbase, *vbase;
  TL tile;
  typename TL::State s;

  __device__ void head(const Args& a, int hh) {
    const int kvh = hh / a.head_tiles, ht = hh % a.head_tiles;
    nh = min(16, a.group - ht * 16);
    head0 = kvh * a.group + ht * 16;
    kbase = a.kc.data + kvh * a.kc.head;
    vbase = a.vc.data + kvh * a.vc.head;
    tile.head(a, kvh);
  }

  __device__ bool live() const { return (int)(threadIdx.x & 15) < nh; }

  // The tiles at at.t0, then.t0, and so on every `step` tokens, before `end`.
  __device__ void tiles(const Args& a, const int32_t* table, int row, const Range& rg, Spot at,
                        Spot then, int step, int32_t end) {
    if (at.t0 >= end) return;
    const T* q = reinterpret_cast<const T*>(a.q) + row * a.q_r +
                 (int64_t)(head0 + (live() ? threadIdx.x & 15 : 0)) * a.q_h;
    if constexpr (TL::kWalks) {
      tile.walk(a, table, q, live(), rg, at, step, end, s);
    } else {
      tile.load_keys(a, kbase, at);
      tile.load_query(a, q, live());
      tile.load_values(a, vbase, at);
      for (;;) {
        f32x4 sc[2];
        tile.scores(sc);
        const bool more = then.t0 < end;
        if (more) tile.load_keys(a, kbase, then);
        tile.add(a, at.t0, rg, sc, s);
        if (!more) break;
        tile.load_values(a, vbase, then);
        at = then;
        then = TL::spot(a, table, at.t0 + step, step);
      }
    }
  }

  // Joins the states of NW waves through LDS ([NW][nh][kPitch] sums, then (m, l)
  // pairs): to the result, or to `part` ([nh][D], then [nh] pairs) if not null.  The
  // sums lose their factor here.
  template <int NW>
  __device__ void join(const Args& a, int row, int wave, float* lds, float* part) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const float l = sum_over_groups(s.l);
    float* ml = lds + NW * nh * kPitch;
    if (live()) {
      if (g == 0) {
        ml[2 * (wave * nh + c)] = s.m;
        ml[2 * (wave * nh + c) + 1] = l;
      }
      float* mine = lds + (wave * nh + c) * kPitch;
#pragma unroll
      for (int b = 0; b < kRuns; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < kRun; j += 4)
            *reinterpret_cast<f32x4*>(mine + TL::run_of(b, r) + j) =
                f32x4{s.acc[b * kRun + j][r], s.acc[b * kRun + j + 1][r],
                      s.acc[b * kRun + j + 2][r], s.acc[b * kRun + j + 3][r]} *
                TL::lower(s);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * (DP / 4); i += 64 * NW) {
      const int h = i / (DP / 4), d = i % (DP / 4) * 4;
      float m = neg_inf();
#pragma unroll
      for (int w = 0; w < NW; ++w) m = fmaxf(m, ml[2 * (w * nh + h)]);
      const float m0 = m == neg_inf() ? 0.0f : m;
      float sum = 0.0f;
      f32x4 o = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = exp_of<T>(ml[2 * (w * nh + h)] - m0);
        sum += f * ml[2 * (w * nh + h) + 1];
        o += f * *reinterpret_cast<const f32x4*>(lds + (w * nh + h) * kPitch + d);
      }
      if (part) {
        if (d < a.D) *reinterpret_cast<f32x4*>(part + h * a.D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(part + nh * a.D + 2 * h) = float2{m, sum};
      } else {
        const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
        const float v[4] = {o[0] * scale, o[1] * scale, o[2] * scale, o[3] * scale};
        store_run<T, 4, TL::kLimit>(a, row, head0 + h, d, v);
        if (d == 0) store_lse(a, row, head0 + h, m, sum);
      }
    }
  }
};

// The item of a workgroup.  Consecutive workgroups go to the eight XCDs in turn, so the
// head tiles of one key/value head come eight apart: they find its keys and values in
// the same L2 (32 requests of 8000 tokens, one key/value head of 128, bf16: 128 query
// heads 159 us with neighbouring workgroups, 91 so; 32 heads 53 and 41).
__device__ inline int item_of(int block, int blocks, int together) {
  if (together == 1) return block;
  const int first = block / (8 * together) * 8;   // of the key/value heads
  const int wide = min(8, blocks / together - first), o = block - first * together;
  return (first + o % wide) * together + o / wide;
}

// NW waves to an item (row, key/value head, head tile); with one, a workgroup's
// four waves have four items.  Eight waves against a wave to an item, key/value heads
// of 64, bf16, in us: 64 requests of up to 256 tokens with 4 heads 5.8 and 12.1, 4096 of
// up to 512 268 and 223; f32, one request of 300 tokens with 8 heads: 9.1 and 28.7.
template <typename TL, int NW>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW, NW == 1 ? TL::kAloneWaves : 1)
void attn_kernel(typename TL::Args a) {
  typedef Attend<TL> A;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = NW == 1 ? (int)blockIdx.x * 4 + wave
                           : item_of(blockIdx.x, gridDim.x, TL::together(a));
  if (NW == 1 && item >= a.items) return;
  const int all = a.kv_heads * a.head_tiles, row = item / all;
  A at;
  at.head(a, item % all);
  at.s.reset();
  const int32_t* table = a.tables + row * a.table_stride;
  constexpr int kStep = NW * TL::kTokens;
  const int32_t mine = (NW == 1 ? 0 : wave) * TL::kTokens;
  Spot first{mine, 0}, second{mine + kStep, 0};
  if (a.window == 0 && a.width > 0) {   // the first pages are asked for along with the length
    first = TL::spot(a, table, mine, kStep);
    second = TL::spot(a, table, mine + kStep, kStep);
  }
  const Range rg = attn_range_uniform(a, row, TL::kTokens);
  if (a.window && a.width > 0) {
    first = TL::spot(a, table, rg.base + mine, kStep);
    second = TL::spot(a, table, rg.base + mine + kStep, kStep);
  }
  at.tiles(a, table, row, rg, first, second, kStep, rg.hi);
  if constexpr (NW > 1) {
    extern __shared__ float lds[];
    at.template join<NW>(a, row, wave, lds, nullptr);
  } else {
    const int lane = threadIdx.x & 63, c = lane & 15;
    const float l = sum_over_groups(at.s.l);
    if (!at.live()) return;
    const float scale = l == 0.0f ? 0.0f : 1.0f / l * TL::lower(at.s);
#pragma unroll
    for (int b = 0; b < A::kRuns; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float v[A::kRun];
#pragma unroll
        for (int j = 0; j < A::kRun; ++j) v[j] = at.s.acc[b * A::kRun + j][r] * scale;
        store_run<typename TL::Type, A::kRun, TL::kLimit>(a, row, at.head0 + c, TL::run_of(b, r), v);
      }
    if (lane < 16) store_lse(a, row, at.head0 + c, at.s.m, l);
  }
}

// Steps of a row: at least one, so that every row's output is written.
template <int STEP>
__device__ inline int row_steps(const Range& rg) {
  return rg.hi > rg.base ? (rg.hi - rg.base + STEP - 1) / STEP : 1;
}

// Steps of a range, for `total` steps in all.
__device__ inline int range_steps(const AttnArgs& a, int total) {
  return max((total + a.ranges - 1) / a.ranges, min(kLeastSteps, total / a.rows));
}

// Floats of a part's place: D values, m and l for each head of a tile, up to a whole number
// of 16 bytes (which an odd number of heads does not make), since parts are accessed 16
// bytes at a time.
__host__ __device__ inline int part_floats(int group, int D) {
  return ((group < 16 ? group : 16) * (D + 2) + 3) & ~3;
}

// Where a part goes: a workgroup has two places, for the row that began in an
// earlier range (or with the range) and for one that begins inside it.
__device__ inline float* part_at(const AttnArgs& a, int range, int hh, bool inside) {
  const int64_t slot = ((int64_t)range * a.kv_heads * a.head_tiles + hh) * 2 + inside;
  return a.part + slot * part_floats(a.group, a.D);
}

template <typename TL>
__global__ __launch_bounds__(64 * kRangeWaves, TL::kRangeOnSimd)
void attn_range_kernel(typename TL::Args a) {
  typedef Attend<TL> A;
  constexpr int kTile = TL::kTokens, kStep = kRangeWaves * kTile, kThreads = 64 * kRangeWaves;
  extern __shared__ float lds[];
  int32_t* scan = reinterpret_cast<int32_t*>(lds);   // before the first join needs it
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int all = a.kv_heads * a.head_tiles;
  const int item = item_of(blockIdx.x, gridDim.x, TL::together(a));
  const int range = item / all, hh = item % all;
  // prefix sums of the rows' steps: a thread has `per` neighbouring rows
  const int per = (a.rows + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, a.rows), r1 = min(r0 + per, a.rows);
  int sum = 0;
  for (int r = r0; r < r1; ++r) sum += row_steps<kStep>(attn_range(a, r, kTile));
  int upto = sum;
  for (int x = 1; x < 64; x <<= 1) {
    const int y = __shfl_up(upto, x);
    if (lane >= x) upto += y;
  }
  if (lane == 63) scan[wave] = upto;
  __syncthreads();
  int total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kRangeWaves; ++w) {
    if (w < wave) before += scan[w];
    total += scan[w];
  }
  int at = before + upto - sum;                      // of row r0
  const int q = range_steps(a, total);
  int x = __builtin_amdgcn_readfirstlane(range * q);
  const int x1 = __builtin_amdgcn_readfirstlane(min(x + q, total));
  if (x >= x1) return;                               // (the first workgroup never)
  for (int r = r0; r < r1; ++r) {
    const int n = row_steps<kStep>(attn_range(a, r, kTile));
    if (at <= x && x < at + n) {
      scan[8] = r;
      scan[9] = at;
    }
    if (blockIdx.x == 0) {
      a.prefix[r] = at;
      if (r == a.rows - 1) a.prefix[a.rows] = at + n;
    }
    at += n;
  }
  __syncthreads();
  int row = __builtin_amdgcn_readfirstlane(scan[8]);
  int start = __builtin_amdgcn_readfirstlane(scan[9]);
  __syncthreads();
  A s;
  s.head(a, hh);
  Range rg = attn_range_uniform(a, row, kTile);
  for (bool first = true;; first = false) {
    const int n = row_steps<kStep>(rg);
    const int from = x - start, to = min(n, x1 - start);
    const int32_t* table = a.tables + row * a.table_stride;
    const int32_t t0 = rg.base + from * kStep + wave * kTile;
    const int32_t end = min(rg.hi, rg.base + to * kStep);
    Spot one{t0, 0}, two{t0 + kStep, 0};
    if (a.width > 0) {
      one = TL::spot(a, table, t0, kStep);
      two = TL::spot(a, table, t0 + kStep, kStep);
    }
    s.s.reset();
    s.tiles(a, table, row, rg, one, two, kStep, end);
    const bool whole = from == 0 && to == n;
    s.template join<kRangeWaves>(a, row, wave, lds,
                                 whole ? nullptr : part_at(a, range, hh, !first));
    x = start + to;
    if (x >= x1) return;
    __syncthreads();                                 // the joined states have been read
    start += n;
    ++row;
    rg = attn_range_uniform(a, row, kTile);
  }
}

// Joins the parts of every (row, head) that lies in several ranges.  LANES lanes
// have a head's values, four neighbouring ones each; `ways` such groups share a
// head's parts, taken in turn, and are joined in their order.  Bound by latency: 6.6 us
// behind 256 ragged requests (8192 heads, most with one or two parts), 8.8 us behind
// three long ones (192 heads of some 40 parts).
template <typename TL>
__global__ __launch_bounds__(256) void join_kernel(typename TL::Args a, int ways) {
  typedef typename TL::Type T;
  constexpr int LANES = TL::kDP / 4;
  constexpr int kGroups = 256 / LANES;
  __shared__ f32x4 sums[kGroups][LANES];
  __shared__ float2 stats[kGroups];
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, way = group % ways;
  const int64_t rh = (int64_t)blockIdx.x * (kGroups / ways) + group / ways;
  bool in = rh < (int64_t)a.rows * a.heads;
  const int row = in ? (int)(rh / a.heads) : 0, head = in ? (int)(rh % a.heads) : 0;
  const int q = range_steps(a, a.prefix[a.rows]);
  const int p0 = a.prefix[row], first = p0 / q, last = (a.prefix[row + 1] - 1) / q;
  in = in && first != last;
  const int n = in ? last - first + 1 : 0;
  const int kvh = head / a.group, ht = head % a.group / 16, c = head % a.group % 16;
  const int hh = kvh * a.head_tiles + ht, nh = min(16, a.group - ht * 16);
  const int d = lane * 4;
  const auto place = [&](int s) { return part_at(a, first + s, hh, s == 0 && p0 > first * q); };
  float m = neg_inf();
#pragma unroll 4
  for (int s = way; s < n; s += ways) m = fmaxf(m, place(s)[nh * a.D + 2 * c]);
  float m0 = m == neg_inf() ? 0.0f : m;
  float sum = 0.0f;
  f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = way; s < n; s += ways) {
    const float* p = place(s);
    const float f = exp_of<T>(p[nh * a.D + 2 * c] - m0);
    sum += f * p[nh * a.D + 2 * c + 1];
    if (d < a.D) o += f * *reinterpret_cast<const f32x4*>(p + c * a.D + d);
  }
  if (ways > 1) {
    sums[group][lane] = o;
    if (lane == 0) stats[group] = float2{m, sum};
    __syncthreads();
    if (way) return;
    for (int w = 1; w < ways; ++w) m = fmaxf(m, stats[group + w].x);
    m0 = m == neg_inf() ? 0.0f : m;
    sum = 0.0f;
    o = f32x4{0, 0, 0, 0};
    for (int w = 0; w < ways; ++w) {
      const float f = exp_of<T>(stats[group + w].x - m0);
      sum += f * stats[group + w].y;
      o += f * sums[group + w][lane];
    }
  }
  if (!in) return;
  const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
  const float v[4] = {o[0] * scale, o[1] * scale, o[2] * scale, o[3] * scale};
  store_run<T, 4, TL::kLimit>(a, row, head, d, v);
  if (lane == 0) store_lse(a, row, head, m, sum);
}

}  // namespace ctcpb_lm
