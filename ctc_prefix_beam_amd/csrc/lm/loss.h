// Token losses over a vocabulary without keeping the logits, and their
// gradients.
//
// Forward: logit tiles (vocabulary x tokens) are computed by gemm_kernel and
// leave it only as a maximum and a sum of exponentials per token and tile;
// loss_join_kernel joins them.  Backward: a piece of the vocabulary at a time,
//   d[n, v] = g[n] (exp(logit[n, v] - lse[n]) - [v = t[n]])
// is recomputed, rounded to the inputs' type and kept for the piece only (at most
// kPieceBytes of workspace, or 256 labels); dx += d w and dw = d^T x follow from it.
//
// The rounding of d to 16 bits adds to dx and dw about what their own rounding to that
// type does.  d is scaled so that the largest |g| is a power of two: the targets' entries,
// -g (1 - p), the largest of their rows, then lie just below one where rows share that
// weight, where a rounding is smallest for its number; with f16 it also keeps d in range.
// Errors of dx and dw over those of rounding the exact results, bf16, 300 to 4096 tokens
// and 500 to 20000 labels: equal weights 1.02 to 1.23, weights spread evenly over [-1, 1]
// 1.33 to 1.39, over a factor of 400 1.36 to 1.45; weights of 1 (2 % of the rows) and 0.51,
// whose targets' entries are all rounded the same way, 1.8 to 2.2.
//
// With up to kPairRows tokens or kPairWork multiplications, where errors average least, and
// wherever the caller asks for it, d is kept as the sum of two values of the type in neighbouring rows (2n and 2n + 1):
// 1.00 in all of these cases, for twice the products of dx and dw, which in small calls wait
// for memory (8192 x 50000 x 2048 bf16: 4.04 and 7.25 ms, 20000 x 5000 x 1024: 0.63 and 0.96).
#pragma once
#include "gemm.h"

namespace ctcpb_lm {

// What the logit epilogues share.
struct Logits {
  const float* bias;        // or null
  const int32_t* targets;
  int32_t tokens, vocab;
  int32_t v0;               // first vocabulary row of the launch
};

// Adds the bias of a wave's rows i*16 + r (`bias`: of the first of them, in LDS).
template <int TM, int TN>
__device__ inline void add_bias(f32x4 (&acc)[TM][TN], const float* bias) {
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const f32x4 b = *reinterpret_cast<const f32x4*>(bias + i * 16);
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] += b;
  }
}

// The loss is bound by the matrix product, and then by the exponentials of its epilogue,
// which the matrix units wait for (a quarter-rate instruction for each logit): 20000 x
// 5000 x 1024 bf16 192 us a call (187 to 199 from card to card), 1070 TFLOP/s, of which 166
// without the epilogue (in a copy) where the whole took 187; 8192 x 50000 x 2048 1.26 to 1.36
// ms, 1330 to 1230 TFLOP/s, and 1.24 where it took 1.36.  The matrix units are
// busy in 63 % of the cycles of the latter.
//
// The epilogues of the logits run with the next item's fetches under way, which
// would delay loads of their own: what they need of the item's rows and columns is
// fetched into LDS with its first tiles ([BM] bias, then arrays of [BN]).
struct ForwardEpilogue {
  Logits lg;
  float2* part;             // [vocabulary tile][token]: maximum, sum of exp(logit - maximum)
  float* hit;               // [token]: logit of the target

  static constexpr bool kJoins = true;
  template <int BM, int BN>
  static constexpr int wanted() {
    return BM + BN;
  }
  template <int BM, int BN, int W>
  __device__ void fetch(const Place& at, float* to, int wave, int lane) const {
    if (lg.bias)
      fetch_floats<BM, W>(lg.bias + at.m * BM, lg.vocab - at.m * BM, to, 0, wave, lane);
    fetch_floats<BN, W>(lg.targets + at.n0, lg.tokens - at.n0, to + BM, BM / 64, wave, lane);
  }

  template <int TM, int TN, int WM, int WN>
  __device__ void run(f32x4 (&acc)[TM][TN], const Place& at, int wm, int wn, int lane,
                      float2* red, const float* got) {
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    const int g = lane >> 4, c = lane & 15;
    const int vb = (at.m * WM + wm) * TM * 16 + g * 4;
    if (lg.bias) add_bias<TM, TN>(acc, got + wm * TM * 16 + g * 4);
    if ((at.m * WM + wm + 1) * TM * 16 > lg.vocab) {   // rows past the vocabulary
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            if (vb + i * 16 + r >= lg.vocab) acc[i][j][r] = neg_inf();
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int k = (wn * TN + j) * 16 + c, n = at.n0 + k;
      const int t = n < lg.tokens ? __float_as_int(got[BM + k]) : -1;
      if (__any(t >= vb && t < vb + TM * 16 && t < lg.vocab)) {   // few tiles have a target
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (vb + i * 16 + r == t && t < lg.vocab) hit[n] = acc[i][j][r];
      }
      float m = neg_inf();
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
      m = max_over_groups(m);
      const float m0 = m == neg_inf() ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) s += exp_fast(acc[i][j][r] - m0);
      s = sum_over_groups(s);
      if (g == 0) red[wm * BN + (wn * TN + j) * 16 + c] = float2{m, s};
    }
    __syncthreads();
    for (int k = threadIdx.x; k < BN; k += 64 * WM * WN) {
      const int n = at.n0 + k;
      if (n >= lg.tokens) continue;
      float m = neg_inf(), s = 0.0f;
      for (int w = 0; w < WM; ++w) m = fmaxf(m, red[w * BN + k].x);
      const float m0 = m == neg_inf() ? 0.0f : m;
      for (int w = 0; w < WM; ++w) s += red[w * BN + k].y * exp_fast(red[w * BN + k].x - m0);
      part[(int64_t)at.m * lg.tokens + n] = float2{m, s};
    }
  }
};

// Joins the tiles of TOKENS tokens, 256 / TOKENS threads to each.  Tokens from
// `main` on were cut into other tiles.  Four tokens to a workgroup where there are few
// (32 tokens of 79 tiles: 3.1 us), 32 where there are many (20000 tokens of 20 tiles:
// 4.6 us, of which reading the 3.2 MB takes one).
template <int TOKENS>
__global__ __launch_bounds__(256) void loss_join_kernel(const float2* part, const float* hit,
                                                        const int32_t* targets, int32_t tokens,
                                                        int32_t vocab, int32_t main, int32_t tiles,
                                                        int32_t rest_tiles, float* loss,
                                                        float* lse) {
  constexpr int kShare = 256 / TOKENS;
  __shared__ float2 red[kShare][TOKENS + 1];
  const int c = threadIdx.x % TOKENS, k = threadIdx.x / TOKENS;
  const int64_t n = (int64_t)blockIdx.x * TOKENS + c;
  float m = neg_inf(), s = 0.0f;
  if (n >= main) tiles = rest_tiles;
  if (n < tokens)
#pragma unroll 4
    for (int t = k; t < tiles; t += kShare) {
      const float2 p = part[t * (int64_t)tokens + n];
      const float m1 = fmaxf(m, p.x), m0 = m1 == neg_inf() ? 0.0f : m1;
      s = s * expf(m - m0) + p.y * expf(p.x - m0);
      m = m1;
    }
  red[k][c] = float2{m, s};
  __syncthreads();
  for (int half = kShare / 2; half; half >>= 1) {
    if (k < half) {
      const float2 p = red[k][c], q = red[k + half][c];
      const float m1 = fmaxf(p.x, q.x), m0 = m1 == neg_inf() ? 0.0f : m1;
      red[k][c] = float2{m1, p.y * expf(p.x - m0) + q.y * expf(q.x - m0)};
    }
    __syncthreads();
  }
  if (k || n >= tokens) return;
  const float l = red[0][c].x + logf(red[0][c].y);
  const int t = targets[n];
  lse[n] = l;
  loss[n] = t >= 0 && t < vocab ? l - hit[n] : 0.0f;
}

// d of one piece of the vocabulary, and the piece's partial sums for dbias.  Bound as
// the loss is, and by writing d: 8192 x 50000 x 2048 bf16 1.45 ms, 1155
// TFLOP/s, matrix units busy in 55 % of the cycles.
template <typename T>
struct GradEpilogue {
  Logits lg;
  const float *grad, *lse;
  const float* scale;       // what d is multiplied by, or null
  T* d;                     // [token][ldd], with pairs [2 token]
  bool pairs;
  int64_t ldd;
  float* dbias_part;        // [token tile and wave][rows], or null
  int32_t rows;             // vocabulary rows of the piece
  int32_t first_part;       // of this launch

  static constexpr bool kJoins = false;
  template <int BM, int BN>
  static constexpr int wanted() {
    return BM + 3 * BN;
  }
  template <int BM, int BN, int W>
  __device__ void fetch(const Place& at, float* to, int wave, int lane) const {
    const int v = lg.v0 + at.m * BM, n = lg.tokens - at.n0;
    if (lg.bias) fetch_floats<BM, W>(lg.bias + v, lg.vocab - v, to, 0, wave, lane);
    fetch_floats<BN, W>(lg.targets + at.n0, n, to + BM, BM / 64, wave, lane);
    fetch_floats<BN, W>(lse + at.n0, n, to + BM + BN, (BM + BN) / 64, wave, lane);
    fetch_floats<BN, W>(grad + at.n0, n, to + BM + 2 * BN, (BM + 2 * BN) / 64, wave, lane);
  }

  template <int TM, int TN, int WM, int WN>
  __device__ void run(f32x4 (&acc)[TM][TN], const Place& at, int wm, int wn, int lane, float2*,
                      const float* got) {
    constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
    const int g = lane >> 4, c = lane & 15;
    const int vl = (at.m * WM + wm) * TM * 16 + g * 4;   // in the piece
    const int vb = lg.v0 + vl;
    const float sc = scale ? scale[0] : 1.0f, inv = scale ? scale[1] : 1.0f;
    if (lg.bias) add_bias<TM, TN>(acc, got + wm * TM * 16 + g * 4);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int k = (wn * TN + j) * 16 + c, n = at.n0 + k;
      const bool live = n < lg.tokens;
      const int t = live ? __float_as_int(got[BM + k]) : -1;
      const bool in = t >= 0 && t < lg.vocab;
      // a row without a target has d = 0, whatever its logits are
      const float gn = in ? sc * got[BM + 2 * BN + k] : 0.0f;
      const float ln = got[BM + BN + k];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = in ? gn * exp_of<T>(acc[i][j][r] - ln) : 0.0f;
      if (__any(in && t >= vb && t < vb + TM * 16)) {   // few tiles have a target
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (in && vb + i * 16 + r == t) acc[i][j][r] -= gn;
      }
      if (vb + TM * 16 > lg.vocab) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (vb + i * 16 + r >= lg.vocab) acc[i][j][r] = 0.0f;
      }
      T* row = d + (pairs ? 2 * n : n) * ldd + (at.m * WM + wm) * TM * 16;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < TM; i += 2) {
          const f32x4 x = acc[i][j], y = acc[i + 1][j];
          const TilePair<T> hi(x, y);
          if (live) hi.store(row + i * 16 + TilePair<T>::at(g));
          if (pairs) {
            f32x4 xl, yl;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              xl[r] = x[r] - (float)(T)x[r];
              yl[r] = y[r] - (float)(T)y[r];
            }
            const TilePair<T> lo(xl, yl);
            if (live) lo.store(row + ldd + i * 16 + TilePair<T>::at(g));
          }
        }
      } else if (live) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
          *reinterpret_cast<f32x4*>(row + i * 16 + g * 4) = acc[i][j];
      }
    }
    if (!dbias_part) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < TN; ++j) s += acc[i][j][r];   // rows past the tokens are 0
        for (int x = 1; x < 16; x <<= 1) s += __shfl_xor(s, x);
        const int v = vl + i * 16 + r;
        if (c == 0 && v < rows)
          dbias_part[(int64_t)(first_part + at.n * WN + wn) * rows + v] = s * inv;
      }
  }
};

// Adds the token tiles' partial sums of a piece, in their order (28 tiles of 5000 entries
// 4.2 us: latency, with eight loads under way at a time; 8 us one after another).
__global__ __launch_bounds__(256) void dbias_kernel(const float* part, int32_t parts, int32_t vocab,
                                                    float* dbias) {
  const int v = blockIdx.x * 256 + threadIdx.x;
  if (v >= vocab) return;
  float s = 0.0f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) s += part[(int64_t)p * vocab + v];
  dbias[v] = s;
}

// Where the sums of a launch go: out[n, m] (m contiguous), rounded, or float32
// `sums`, added to what earlier pieces of the vocabulary left there (`add`);
// with k in parts, each part's sums to a plane of its own, [the launch's rows][M].  The products are bound by
// the matrix units, busy in 65 % (dx) and 67 % (dw) of the cycles at 8192 x 50000 x 2048
// bf16: 1.25 and 1.30 ms, 1345 and 1290 TFLOP/s.
template <typename T>
struct OutEpilogue {
  T* out;
  float *sums, *planes;     // or null
  int64_t from, pitch;      // of the planes: the value of the result that each begins with, and
                            // the values of one
  const float* scale;       // what d was multiplied by, or null
  int32_t M, N;
  bool pairs;               // the product's rows n = 2i and 2i + 1 add up to row i
  bool add, last;           // sums hold something; the result goes to `out`

  static constexpr bool kJoins = false;
  template <int BM, int BN>
  static constexpr int wanted() {
    return 0;
  }
  template <int BM, int BN, int W>
  __device__ void fetch(const Place&, float*, int, int) const {}

  template <int TM, int TN, int WM, int WN>
  __device__ void run(f32x4 (&acc)[TM][TN], const Place& at, int wm, int wn, int lane, float2*,
                      const float*) {
    const int g = lane >> 4, c = lane & 15;
    const int mb = (at.m * WM + wm) * TM * 16 + g * 4;
    const float inv = scale ? scale[1] : 1.0f;
    float* f = planes ? planes : last ? nullptr : sums;
    const int64_t shift = planes ? at.split * pitch - from : 0;   // of f's values
    // results of 16-bit types whose rows are 16-byte aligned
    const bool wide = sizeof(T) == 2 && !f && M % 8 == 0;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      int n = at.n0 + (wn * TN + j) * 16 + c;
      bool live = true;
      if (pairs) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] += __shfl_xor(acc[i][j][r], 1);
        live = !(c & 1);
        n >>= 1;
      }
      live = live && n < N;
      if (add && live) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (mb + i * 16 + r < M) acc[i][j][r] += sums[(int64_t)n * M + mb + i * 16 + r];
      }
      if constexpr (sizeof(T) == 2) {
        if (wide) {
#pragma unroll
          for (int i = 0; i < TM; i += 2) {
            const TilePair<T> t(acc[i][j] * inv, acc[i + 1][j] * inv);
            const int m = mb - g * 4 + i * 16 + TilePair<T>::at(g);
            if (live && m < M) t.store(out + (int64_t)n * M + m);
          }
          continue;
        }
      }
      if (!live) continue;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int m = mb + i * 16;
        const int64_t to = (int64_t)n * M + m;
        if (f && M % 4 == 0) {   // rows start 4-element aligned: four values or none
          if (m < M) *reinterpret_cast<f32x4*>(f + (to + shift)) = acc[i][j];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (m + r >= M) continue;
            if (f)
              f[to + shift + r] = acc[i][j][r];
            else
              out[to + r] = (T)(acc[i][j][r] * inv);
          }
        }
      }
    }
  }
};

// Adds `count` planes of n values, in their order, to `before` (if
// not null: what earlier pieces of the vocabulary left) and leaves the result in
// `sums` or, rounded, in `out`.  Bound by memory: 4 planes of 875 x 384 4.8 us, 2 of
// 848 x 2048 6.9 us.
template <typename T>
__global__ __launch_bounds__(256) void planes_kernel(const float* planes, int32_t count, int64_t n,
                                                     const float* before, float* sums, T* out,
                                                     const float* scale) {
  const float inv = scale ? scale[1] : 1.0f;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    float v = before ? before[i] : 0.0f;
#pragma unroll 4
    for (int p = 0; p < count; ++p) v += planes[p * n + i];
    if (sums)
      sums[i] = v;
    else
      out[i] = (T)(v * inv);
  }
}

// scale[0]: what takes the largest |grad| of a row with a target to `top`, a power
// of two, and scale[1] its inverse.  One workgroup, since the largest of all is asked
// for: 5.8 us for 8192 rows, in front of milliseconds.
__global__ __launch_bounds__(1024) void scale_kernel(const float* grad, const int32_t* targets,
                                                     int32_t tokens, int32_t vocab, float top,
                                                     float* scale) {
  __shared__ float most[16];
  float m = 0.0f;
  for (int64_t n0 = threadIdx.x; n0 < tokens; n0 += 8 * 1024) {
    float v[8];
    int32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // all of them on their way at once
      const int64_t n = n0 + i * 1024;
      v[i] = n < tokens ? grad[n] : 0.0f;
      t[i] = n < tokens ? targets[n] : -1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t[i] >= 0 && t[i] < vocab && fabsf(v[i]) <= 3.4028235e38f) m = fmaxf(m, fabsf(v[i]));
  }
  for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 0; w < 16; ++w) m = fmaxf(m, most[w]);
  const float s = m > 0.0f ? fminf(fmaxf(top / m, 1e-30f), 1e30f) : 1.0f;
  scale[0] = s;
  scale[1] = 1.0f / s;
}

}  // namespace ctcpb_lm
