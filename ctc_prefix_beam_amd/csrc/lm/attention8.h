// Attention of one token per request over a paged cache held in 8 bits, with a scale for
// each page and head: k_t = scale_k[page of t] code_k[t], v_t alike.
//
// The kernels are those of attention.h (short requests, ranges, join) with another tile.  What
// is read is half of a 16-bit cache, so what each value costs beside its load counts twice:
//
// - Both products are f16 ones.  Every code is an f16 value (of whole numbers, 1/512 of it), so
//   the cache enters them without a rounding; widening a pair costs 1 or 2.5 instructions.
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
// Layout of a tile of 32 tokens: as for 16-bit types, but a lane (g, c) has 16 bytes of a key's row at
// d = 64 k + 16 g (which two k-steps of the product take in that order, q alike) and, of the
// values of tokens 8g .. 8g+7, DP / 16 bytes at d = c DP / 16.
#pragma once
#include "attention.h"
#include "cache8.h"

namespace ctcpb_lm {

struct Attn8Args : AttnArgs {
  ScaleView ks, vs;
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
  static constexpr int kAloneWaves = DP <= 128 ? 4 : 2;
  static constexpr int kRangeOnSimd = DP <= 128 ? 4 : 2;
  static constexpr int kTokens = 32;
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
  uint32_t vr[8][kV / 4];
  const float *kscales, *vscales;
  float kscale, vscale;   // of the lane's group of four tokens
  float qscale;

  __device__ void head(const Args& a, int kvh) {
    kscales = a.ks.data + kvh * a.ks.head;
    vscales = a.vs.data + kvh * a.vs.head;
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
          typedef T TN __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
          for (int v = 0; v < (int)sizeof(T) / 2; ++v) {
            const TN y = reinterpret_cast<const TN*>(src + d)[v];
#pragma unroll
            for (int i = 0; i < 16 / (int)sizeof(T); ++i) x[k][v * (16 / (int)sizeof(T)) + i] = y[i];
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

  static __device__ Spot spot(const Args& a, const int32_t* table, int32_t t0) {
    return Spot{t0, group_page(a, table, t0 + (threadIdx.x & 7) * 4)};
  }

  __device__ void load_keys(const Args& a, const char* base, const Spot& at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    kscale = kscales[at.page * a.ks.page];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int grp = (c >> 2) * 2 + h;
      const int64_t page = __shfl(at.page, grp);
      const int32_t t = at.t0 + grp * 4 + (c & 3);
      const char* p = base + page * a.kc.page + (int64_t)(t & mask) * a.kc.token;
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        const int d = k * 64 + g * 16;
        kf[h][k] = u32x4{0, 0, 0, 0};
        if (d < a.D) kf[h][k] = *reinterpret_cast<const u32x4*>(p + d);
      }
    }
  }

  __device__ void load_values(const Args& a, const char* base, const Spot& at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int32_t mask = (1 << a.page_log) - 1;
    vscale = vscales[at.page * a.vs.page];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int grp = g * 2 + h;
      const int64_t page = __shfl(at.page, grp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t t = at.t0 + grp * 4 + i;
        const char* p = base + page * a.vc.page + (int64_t)(t & mask) * a.vc.token + c * kV;
        uint32_t (&to)[kV / 4] = vr[h * 4 + i];
#pragma unroll
        for (int x = 0; x < kV / 4; ++x) to[x] = 0;
        if (c * kV < a.D) {
          if constexpr (kV == 16) {
            const u32x4 z = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int x = 0; x < 4; ++x) to[x] = z[x];
          } else if constexpr (kV == 8) {
            const u32x2 z = *reinterpret_cast<const u32x2*>(p);
            to[0] = z[0];
            to[1] = z[1];
          } else {
            to[0] = *reinterpret_cast<const uint32_t*>(p);
          }
        }
      }
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

  // Scores of the lane's eight tokens t0 + 8g .. for head c.
  __device__ void scores(f32x4 (&sc)[2]) const {
    const int g = (threadIdx.x & 63) >> 4;
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
      sc[h] *= __shfl(kscale, g * 2 + h) * qscale;
    }
  }

  __device__ void add(const Args& a, int32_t t0, const Range& rg, const f32x4 (&sc)[2], State& s) {
    const int g = (threadIdx.x & 63) >> 4;
    const bool whole = t0 >= rg.lo && t0 + 32 <= rg.hi;
    const float scale[2] = {__shfl(vscale, g * 2), __shfl(vscale, g * 2 + 1)};
    float p[8], w[8];
    float top = neg_inf();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = sc[i >> 2][i & 3];
      w[i] = scale[i >> 2];
      if (!whole) {
        const int32_t t = t0 + g * 8 + i;
        if (t < rg.lo || t >= rg.hi) {
          p[i] = neg_inf();
          // a masked slot may hold anything, as may its page's scale, and 0 * NaN is NaN
          w[i] = 0.0f;
#pragma unroll
          for (int x = 0; x < kV / 4; ++x) vr[i][x] = 0;
        }
      }
      top = fmaxf(top, p[i]);
    }
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
#pragma unroll
      for (int i = 0; i < 8; ++i) vr[i][x] = C::prepared(vr[i][x]);
      add_four<0>(x, change, hi, lo, s);
      add_four<2>(x, change, hi, lo, s);
    }
  }

  // Two of a word's values (J and J + 1) of the eight tokens.
  template <int J>
  __device__ void add_four(int x, float change, const f16x8& hi, const f16x8& lo, State& s) {
    f16x2 v[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x2 two[2];
      C::template across<J>(vr[2 * i][x], vr[2 * i + 1][x], two);
      v[0][i] = two[0];
      v[1][i] = two[1];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f16x8 vf = __builtin_bit_cast(f16x8, v[j]);
      f32x4& acc = s.acc[4 * x + J + j];
      f32x4 o = acc * change;
      o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, hi, o, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, lo, o, 0, 0, 0);
    }
  }
};

}  // namespace ctcpb_lm
