// Attention of one token per request over a paged cache held in 8 bits, with a scale for
// each page and head: k_t = scale_k[page of t] code_k[t], v_t alike.
//
// The kernels are those of attention.h (short requests, ranges, join) with another tile.  What
// is read is half of a 16-bit cache, so what each value costs beside its load counts twice:
//
// - Both products are f16 ones.  Every code is an f16 value (of whole numbers, 1/512 of it), so
//   the cache enters them without a rounding; widening a pair costs 1 (e4m3) or 2.5 instructions.
// - q enters as f16 too.  bf16 and f32 ones are first multiplied by the power of two that takes
//   the largest of the head to 2^14 .. 2^15: what of a bf16 value is then lost lies 2^-39 below the
//   largest, less than its float32 product's rounding.  f32 ones are the sum of two f16 values.
// - A score is the codes' product times one number for each four tokens, scale_k times what
//   was taken out of q.
// - The weights of the second product are w_t = p_t scale_v[t], p_t = exp(s_t - m), as the sum of
//   two f16 values, 22 bits.  f16 reaches from 2^-24 to 2^16, scales much farther: w is
//   multiplied by the power of two `up` that takes the largest of the head's weights so far
//   (`top`, which shrinks as m grows) to 2^14 .. 2^15, so that pages of very different scales, and
//   long tails, keep their digits.  The sums acc carry the same factor.
//
// - A wave looks pages and scales up for eight tiles at a time, well before it needs them; what
//   is left to a tile is one multiplication for each group of four tokens' address.  With a
//   lookup for each tile, and addresses multiplied out in 64 bits, 4096 requests of up to 512
//   tokens took 155 us, not 131.
//
// What bounds it, measured: memory.  256 requests of 1..4095 tokens, 32 query and 8 key/value
// heads of 128, int8, bf16: 1.08 GB in 209 us, 5.2 TB/s (a copy: 5.0; 16-bit caches 420 us), the
// matrix units busy in 10 % of the cycles; three requests of up to 131071 tokens, e4m3: 604 MB in
// 119 us, 5.1 TB/s; 4096 requests of up to 512 tokens, 4 heads of 64, e4m3, f16: 542 MB in 131 us
// token by token and 121 head by head (full rows: 5.1 TB/s; the rest is the start and end of
// short ones).  Four waves a SIMD for heads of 128 spill (302 us for the 256 requests), five for
// heads of 64 too (156 for the 4096); two sets of registers for tiles, to fetch two ahead, leave
// two waves and take 225.  Some of what is kept spills as well, mostly outside the loop over tiles:
// ranges of int8 codes with heads of 64 seven registers; all ranges with f32 q, of which there are
// two halves, 8 to 23; and f32 heads of 256 with a wave to an item 4 and 9.  Inside the loop are up
// to four of 885 instructions, for f32 heads of 256.  256 requests of up to 1024 tokens, 8 heads of
// 64, f32: 51 us for 134 MB, half of a copy's rate.  A tile costs as many vector instructions for
// one query head as for 16.
//
// Layout of a tile of 32 tokens: as for 16-bit types, but a lane (g, c) has 16 bytes of a key's
// row at d = 64 k + 16 g (which two k-steps of the product take in that order, q alike) and, of
// the values of tokens 8g .. 8g+7, DP / 16 bytes at d = c DP / 16.
#pragma once
#include <type_traits>

#include "attention.h"
#include "cache8.h"

namespace ctcpb_lm {

struct Attn8Args : AttnArgs {
  ScaleView ks, vs;
  uint32_t k_page, v_page, k_token, v_token;   // strides of the caches in bytes
  uint32_t ks_page, vs_page;                   // and of the scales in bytes
};

// The power of two that takes a magnitude to 2^14 .. 2^15, between 2^-113 and 2^126.
__device__ inline float to_top(float magnitude) {
  const uint32_t e = max(f32_bits(magnitude) >> 23, 15u);
  return bits_f32((268u - e) << 23);
}
// 1 / u of a power of two that to_top() gave.
__device__ inline float undo(float u) { return bits_f32((254u << 23) - f32_bits(u)); }

template <int NA>
struct WaveState8 {
  float m, l;
  float top, up;    // largest weight, and what weights and sums are multiplied by
  f32x4 acc[NA];

  __device__ void reset() {
    m = neg_inf();
    l = top = 0.0f;
    up = 1.0f;
#pragma unroll
    for (int j = 0; j < NA; ++j) acc[j] = f32x4{0, 0, 0, 0};
  }
};

template <typename T, typename C, int DP>
struct Tile8 {
  typedef T Type;
  typedef Attn8Args Args;
  static constexpr int kDP = DP;
  static constexpr int kAloneWaves = DP == 64 ? 4 : DP == 128 ? 3 : 2;
  static constexpr int kRangeOnSimd = DP == 64 ? 4 : DP == 128 ? 3 : 2;
  static constexpr int kTokens = 32;
  static constexpr bool kWalks = true;
  // code times scale may be 65536 where 65504 was stored
  static constexpr bool kLimit = __is_same(T, _Float16);
  static constexpr int kK = DP / 64;       // 16-byte loads of a key's row for a lane
  static constexpr int kV = DP / 16;       // bytes of a value's row
  static constexpr int kAcc = DP / 16;
  static constexpr int kQ = sizeof(T) == 4 ? 2 : 1;   // f16 values to a number of q
  typedef WaveState8<kAcc> State;

  static __device__ float lower(const State& s) { return C::kUnit * undo(s.up); }
  // heads of a request: their rows may share lines of memory, and their scales do
  static __device__ int together(const Args& a) { return a.kv_heads * a.head_tiles; }

  f16x8 q[kQ][2 * kK];
  u32x4 kf[2][kK];
  typedef uint32_t Row __attribute__((ext_vector_type(kV / 4 > 1 ? kV / 4 : 2)));
  typedef typename std::conditional<kV == 4, uint32_t, Row>::type ValueRow;
  ValueRow vr[8];
  __device__ uint32_t word(int i, int x) const {
    if constexpr (kV == 4)
      return vr[i];
    else
      return vr[i][x];
  }
  float qscale;

  // Where the lane's rows lie in page 0 for a tile at a page's first token: keys of the two
  // products, values of the two groups of four tokens.  A tile's first token is a multiple
  // of 32, so pages of up to 32 tokens differ by the page alone, longer ones also by t0 & mask,
  // the same for all lanes.
  const char *krow[2], *vrow[2];
  const char *kscales, *vscales;

  __device__ void head(const Args& a, int kvh) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    kscales = reinterpret_cast<const char*>(a.ks.data + kvh * a.ks.head);
    vscales = reinterpret_cast<const char*>(a.vs.data + kvh * a.vs.head);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kt = (c >> 2) * 8 + h * 4 + (c & 3), vt = g * 8 + h * 4;
      krow[h] = a.kc.data + kvh * a.kc.head + (kt & mask) * a.kc.token + g * 16;
      // (what lies past the head's values is computed and not kept: any will do)
      vrow[h] = a.vc.data + kvh * a.vc.head + (vt & mask) * a.vc.token +
                (c * kV < a.D ? c * kV : 0);
    }
  }

  // Pages and scales are looked up for eight tiles at a time, eight groups of four tokens to
  // each: lane 8 i + j has those of group j of tile i of the block that begins at t0.  This is the
  // table's entry as it is; it need not wait for the request's length, for what is past the
  // last token is masked whatever its page holds.
  static __device__ Spot spot(const Args& a, const int32_t* table, int32_t t0, int step) {
    const int lane = threadIdx.x & 63;
    const int32_t t = t0 + (lane >> 3) * step + (lane & 7) * 4;
    return Spot{t0, table[min(t >> a.page_log, a.width - 1)]};
  }
  struct Block {
    uint32_t page;
    float kscale, vscale;
  };
  __device__ Block block(const Args& a, int32_t entry) const {
    Block b;
    b.page = min((uint32_t)entry, (uint32_t)(a.num_pages - 1));
    b.kscale = *reinterpret_cast<const float*>(kscales + (uint64_t)b.page * a.ks_page);
    b.vscale = *reinterpret_cast<const float*>(vscales + (uint64_t)b.page * a.vs_page);
    return b;
  }

  // The tiles at at.t0, at.t0 + step and so on before `end`.
  __device__ void walk(const Args& a, const int32_t* table, const T* query, bool live,
                       const Range& rg, Spot at, int step, int32_t end, State& s) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    Block now = block(a, at.page), next = now;
    int32_t t0 = at.t0, entry = 0;
    if (t0 + 8 * step < end) entry = spot(a, table, t0 + 8 * step, step).page;
    const auto of = [&](int tile, int group) { return tile * 8 + group; };
    load_keys(a, __shfl(now.page, of(0, (c >> 2) * 2)), __shfl(now.page, of(0, (c >> 2) * 2 + 1)),
              t0);
    load_query(a, query, live);
    load_values(a, __shfl(now.page, of(0, g * 2)), __shfl(now.page, of(0, g * 2 + 1)), t0);
    for (int i = 0;; i = (i + 1) & 7) {
      f32x4 sc[2];
      scores(sc);
      const float vscale[2] = {__shfl(now.vscale, of(i, g * 2)),
                               __shfl(now.vscale, of(i, g * 2 + 1))};
#pragma unroll
      for (int h = 0; h < 2; ++h) sc[h] *= __shfl(now.kscale, of(i, g * 2 + h)) * qscale;
      const int32_t then = t0 + step;
      const bool more = then < end;
      // the next block's entries have had four tiles to arrive, its scales have four more
      if (i == 3 && t0 + 5 * step < end) next = block(a, entry);
      if (i == 7 && more) {
        now = next;
        if (then + 8 * step < end) entry = spot(a, table, then + 8 * step, step).page;
      }
      const int j = (i + 1) & 7;
      if (more)
        load_keys(a, __shfl(now.page, of(j, (c >> 2) * 2)),
                  __shfl(now.page, of(j, (c >> 2) * 2 + 1)), then);
      add(a, t0, rg, sc, vscale, s);
      if (!more) break;
      load_values(a, __shfl(now.page, of(j, g * 2)), __shfl(now.page, of(j, g * 2 + 1)), then);
      t0 = then;
    }
  }

  __device__ void load_query(const Args& a, const T* src, bool live) {
    const int g = (threadIdx.x & 63) >> 4;
    T x[2 * kK][8];
#pragma unroll
    for (int k = 0; k < 2 * kK; ++k) {
      const int d = (k >> 1) * 64 + g * 16 + (k & 1) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = (T)0.0f;
      if (live && d < a.D) {
        if (a.wide_q) {
          constexpr int M = 16 / (int)sizeof(T);
          typedef T TM __attribute__((ext_vector_type(M)));
#pragma unroll
          for (int v = 0; v < 8 / M; ++v) {
            const TM y = reinterpret_cast<const TM*>(src + d)[v];
#pragma unroll
            for (int i = 0; i < M; ++i) x[k][v * M + i] = y[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] = src[d + i];
        }
      }
    }
    float up = 1.0f;
    qscale = a.scale * C::kUnit;
    if constexpr (!__is_same(T, _Float16)) {
      float most = 0.0f;
#pragma unroll
      for (int k = 0; k < 2 * kK; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf((float)x[k][i]));
      up = to_top(max_over_groups(most));
      qscale *= undo(up);
    }
#pragma unroll
    for (int k = 0; k < 2 * kK; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (__is_same(T, _Float16)) {
          q[0][k][i] = x[k][i];
        } else {
          const float y = (float)x[k][i] * up;
          q[0][k][i] = (_Float16)y;
          if constexpr (kQ == 2) q[1][k][i] = (_Float16)(y - (float)q[0][k][i]);
        }
      }
  }

  static constexpr int kRun = kV;
  static __device__ int run_of(int, int r) {
    return (((threadIdx.x & 63) >> 4) * 4 + r) * kV;
  }

  __device__ void load_keys(const Args& a, uint32_t page0, uint32_t page1, int32_t t0) {
    const int g = (threadIdx.x & 63) >> 4;
    const uint32_t first = (t0 & ((1 << a.page_log) - 1)) * a.k_token;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char* p = krow[h] + (uint64_t)(h ? page1 : page0) * a.k_page + first;
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        // q is zero for what lies past the head's values: any of the row's will do (half of
        // DP is always there, but for the smallest)
        const bool there = (DP > 64 && 2 * k < kK) || k * 64 + g * 16 < a.D;
        const int d = there ? k * 64 : -g * 16;
        kf[h][k] = *reinterpret_cast<const u32x4*>(p + d);
      }
    }
  }

  __device__ void load_values(const Args& a, uint32_t page0, uint32_t page1, int32_t t0) {
    const uint32_t first = (t0 & ((1 << a.page_log) - 1)) * a.v_token;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char* p = vrow[h] + (uint64_t)(h ? page1 : page0) * a.v_page + first;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vr[h * 4 + i] = *reinterpret_cast<const ValueRow*>(p + i * a.v_token);
    }
  }

  // Eight neighbouring codes of a row.
  static __device__ f16x8 widen(uint32_t a, uint32_t b) {
    a = C::prepared(a);
    b = C::prepared(b);
    const f16x2 x[4] = {C::template two<false>(a), C::template two<true>(a),
                        C::template two<false>(b), C::template two<true>(b)};
    return __builtin_bit_cast(f16x8, x);
  }

  // Products of the lane's eight tokens t0 + 8g .. with head c.
  __device__ void scores(f32x4 (&sc)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sc[h] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const f16x8 f = widen(kf[h][k][2 * x], kf[h][k][2 * x + 1]);
#pragma unroll
          for (int y = kQ - 1; y >= 0; --y)
            sc[h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, q[y][2 * k + x], sc[h], 0, 0, 0);
        }
    }
  }

  __device__ void add(const Args& a, int32_t t0, const Range& rg, const f32x4 (&sc)[2],
                      const float (&vscale)[2], State& s) {
    const int g = (threadIdx.x & 63) >> 4;
    float p[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = sc[i >> 2][i & 3];
      w[i] = vscale[i >> 2];
    }
    if (t0 < rg.lo || t0 + 32 > rg.hi) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t t = t0 + g * 8 + i;
        const bool in = t >= rg.lo && t < rg.hi;
        p[i] = in ? p[i] : neg_inf();
        // a masked slot may hold anything, as may its page's scale, and 0 * NaN is NaN
        w[i] = in ? w[i] : 0.0f;
        if (C::kNan) vr[i] = in ? vr[i] : ValueRow(0);
      }
    }
    float top = neg_inf();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, p[i]);
    const float m = fmaxf(s.m, max_over_groups(top));
    const float m0 = m == neg_inf() ? 0.0f : m;   // nothing seen yet: avoid inf - inf
    const float alpha = exp_of<T>(s.m - m0);
    s.m = m;
    s.l *= alpha;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp_of<T>(p[i] - m0);
      s.l += p[i];
      w[i] *= p[i];
      most = fmaxf(most, fabsf(w[i]));
    }
    s.top = fmaxf(s.top * alpha, max_over_groups(most));
    const float up = to_top(s.top);
    const float change = alpha * undo(s.up) * up;
    s.up = up;
    f16x8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = w[i] * up;
      hi[i] = (_Float16)x;
      lo[i] = (_Float16)(x - (float)hi[i]);
    }
#pragma unroll
    for (int x = 0; x < kV / 4; ++x) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = C::prepared(word(i, x));
      add_two<0>(v, &s.acc[4 * x], change, hi, lo);
      add_two<2>(v, &s.acc[4 * x + 2], change, hi, lo);
    }
  }

  // Two of the values of a word (J and J + 1), of eight tokens.
  template <int J>
  static __device__ void add_two(const uint32_t (&w)[8], f32x4* acc, float change, const f16x8& hi,
                                 const f16x8& lo) {
    f16x2 v[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x2 two[2];
      C::template across<J>(w[2 * i], w[2 * i + 1], two);
      v[0][i] = two[0];
      v[1][i] = two[1];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f16x8 vf = __builtin_bit_cast(f16x8, v[j]);
      f32x4 o = acc[j] * change;
      o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, hi, o, 0, 0, 0);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, lo, o, 0, 0, 0);
    }
  }
};

}  // namespace ctcpb_lm
