// Token losses over a vocabulary without keeping the logits, and their
// gradients.
//
// Forward: logit tiles (vocabulary x tokens) are computed by gemm_kernel and
// leave it only as a maximum and a sum of exponentials per token and tile;
// loss_join_kernel joins them.  Backward: a piece of the vocabulary at a time,
//   d[n, v] = g[n] (exp(logit[n, v] - lse[n]) - [v = t[n]])
// is recomputed, rounded to the inputs' type and kept for the piece only (at most
// kPieceBytes of workspace); dx += d w and dw = d^T x follow from it.  The
// rounding of d is unbiased and enters sums of many terms: it adds to dx and dw
// about what their own rounding to that type does.
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

struct ForwardEpilogue {
  Logits lg;
  float2* part;             // [vocabulary tile][token]: maximum, sum of exp(logit - maximum)
  float* hit;               // [token]: logit of the target

  template <int TM, int TN, int WM, int WN>
  __device__ void run(f32x4 (&acc)[TM][TN], int tm, int tn, int wm, int wn, int lane, char* lds) {
    constexpr int BN = WN * TN * 16;
    const int g = lane >> 4, c = lane & 15;
    const int vb = (tm * WM + wm) * TM * 16 + g * 4;
    float2* red = reinterpret_cast<float2*>(lds);   // [WM][BN]; the tiles are done with
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int v = vb + i * 16 + r;
        const bool in = v < lg.vocab;
        const float b = in && lg.bias ? lg.bias[v] : 0.0f;
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j][r] = in ? acc[i][j][r] + b : neg_inf();
      }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = tn * BN + (wn * TN + j) * 16 + c;
      const int t = n < lg.tokens ? lg.targets[n] : -1;
      float m = neg_inf();
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          m = fmaxf(m, acc[i][j][r]);
          if (vb + i * 16 + r == t && t < lg.vocab) hit[n] = acc[i][j][r];
        }
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
      const int n = tn * BN + k;
      if (n >= lg.tokens) continue;
      float m = neg_inf(), s = 0.0f;
      for (int w = 0; w < WM; ++w) m = fmaxf(m, red[w * BN + k].x);
      const float m0 = m == neg_inf() ? 0.0f : m;
      for (int w = 0; w < WM; ++w) s += red[w * BN + k].y * exp_fast(red[w * BN + k].x - m0);
      part[(int64_t)tm * lg.tokens + n] = float2{m, s};
    }
  }
};

// Joins the tiles of 32 tokens, 8 threads to each.
__global__ __launch_bounds__(256) void loss_join_kernel(const float2* part, const float* hit,
                                                        const int32_t* targets, int32_t tokens,
                                                        int32_t vocab, int32_t tiles, float* loss,
                                                        float* lse) {
  __shared__ float2 red[8][32];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + c;
  float m = neg_inf(), s = 0.0f;
  if (n < tokens)
    for (int t = k; t < tiles; t += 8) {
      const float2 p = part[t * (int64_t)tokens + n];
      const float m1 = fmaxf(m, p.x), m0 = m1 == neg_inf() ? 0.0f : m1;
      s = s * expf(m - m0) + p.y * expf(p.x - m0);
      m = m1;
    }
  red[k][c] = float2{m, s};
  __syncthreads();
  if (k || n >= tokens) return;
  for (int w = 1; w < 8; ++w) m = fmaxf(m, red[w][c].x);
  const float m0 = m == neg_inf() ? 0.0f : m;
  s = 0.0f;
  for (int w = 0; w < 8; ++w) s += red[w][c].y * expf(red[w][c].x - m0);
  const float l = m + logf(s);
  const int t = targets[n];
  lse[n] = l;
  loss[n] = t >= 0 && t < vocab ? l - hit[n] : 0.0f;
}

// d of one piece of the vocabulary, and the piece's partial sums for dbias.
template <typename T>
struct GradEpilogue {
  Logits lg;
  const float *grad, *lse;
  const float* scale;       // f16: power of two that d is multiplied by; else null
  T* d;                     // [token][ldd]
  int64_t ldd;
  float* dbias_part;        // [token tile and wave][vocab], or null

  template <int TM, int TN, int WM, int WN>
  __device__ void run(f32x4 (&acc)[TM][TN], int tm, int tn, int wm, int wn, int lane, char*) {
    constexpr int BN = WN * TN * 16;
    const int g = lane >> 4, c = lane & 15;
    const int vl = (tm * WM + wm) * TM * 16 + g * 4;   // in the piece
    const float sc = scale ? scale[0] : 1.0f;
    f32x4 sum[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) sum[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = tn * BN + (wn * TN + j) * 16 + c;
      const bool live = n < lg.tokens;
      const int t = live ? lg.targets[n] : -1;
      const bool in = t >= 0 && t < lg.vocab;
      const float gn = in ? grad[n] : 0.0f, ln = in ? lse[n] : 0.0f;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        T out[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int v = lg.v0 + vl + i * 16 + r;
          const float b = v < lg.vocab && lg.bias ? lg.bias[v] : 0.0f;
          float p = exp_of<T>(acc[i][j][r] + b - ln);
          p = in && v < lg.vocab ? gn * (v == t ? p - 1.0f : p) : 0.0f;
          sum[i][r] += p;
          out[r] = (T)(p * sc);
        }
        if (live) {
          typedef T T4 __attribute__((ext_vector_type(4)));
          *reinterpret_cast<T4*>(d + n * ldd + vl + i * 16) = T4{out[0], out[1], out[2], out[3]};
        }
      }
    }
    if (!dbias_part) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float s = sum[i][r];
        for (int x = 1; x < 16; x <<= 1) s += __shfl_xor(s, x);
        const int v = lg.v0 + vl + i * 16 + r;
        if (c == 0 && v < lg.vocab) dbias_part[(int64_t)(tn * WN + wn) * lg.vocab + v] = s;
      }
  }
};

__global__ __launch_bounds__(256) void dbias_kernel(const float* part, int32_t parts, int32_t vocab,
                                                    float* dbias) {
  const int v = blockIdx.x * 256 + threadIdx.x;
  if (v >= vocab) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += part[(int64_t)p * vocab + v];
  dbias[v] = s;
}

// out[n, m] (m contiguous) from the sums, which over several launches are added
// up in `sums` (float32) and rounded by the last one.
template <typename T>
struct OutEpilogue {
  T* out;
  float* sums;              // [N][M], null when one launch does it all
  const float* scale;       // f16: what d was multiplied by
  int32_t M, N;
  bool first, last;

  template <int TM, int TN, int WM, int WN>
  __device__ void run(f32x4 (&acc)[TM][TN], int tm, int tn, int wm, int wn, int lane, char*) {
    constexpr int BN = WN * TN * 16;
    const int g = lane >> 4, c = lane & 15;
    const int mb = (tm * WM + wm) * TM * 16 + g * 4;
    const float inv = scale ? scale[1] : 1.0f;
    typedef T T4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = tn * BN + (wn * TN + j) * 16 + c;
      if (n >= N) continue;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int m = mb + i * 16;
        const int64_t at = (int64_t)n * M + m;
        if (M % 4 == 0) {   // rows start 4-element aligned: whole or not at all
          if (m >= M) continue;
          f32x4 v = acc[i][j];
          if (!first) v += *reinterpret_cast<const f32x4*>(sums + at);
          if (!last) {
            *reinterpret_cast<f32x4*>(sums + at) = v;
          } else {
            v *= inv;
            *reinterpret_cast<T4*>(out + at) = T4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
          }
        } else {
          for (int r = 0; r < 4; ++r) {
            if (m + r >= M) break;
            float v = acc[i][j][r];
            if (!first) v += sums[at + r];
            if (!last)
              sums[at + r] = v;
            else
              out[at + r] = (T)(v * inv);
          }
        }
      }
    }
  }
};

// f16 only: a power of two that brings the largest |grad| of a row with a
// target to 2^11..2^12, so that d (at most |grad|) neither overflows nor loses
// its small values, and its inverse.
__global__ __launch_bounds__(1024) void scale_kernel(const float* grad, const int32_t* targets,
                                                     int32_t tokens, int32_t vocab, float* scale) {
  __shared__ float top[16];
  float m = 0.0f;
  for (int n = threadIdx.x; n < tokens; n += 1024) {
    const float v = fabsf(grad[n]);
    const int t = targets[n];
    if (t >= 0 && t < vocab && v <= 3.4028235e38f) m = fmaxf(m, v);
  }
  for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 0; w < 16; ++w) m = fmaxf(m, top[w]);
  int e = 0;
  if (m > 0.0f) frexpf(m, &e);          // m < 2^e
  e = min(max(12 - e, -100), 100);
  scale[0] = ldexpf(1.0f, e);
  scale[1] = ldexpf(1.0f, -e);
}

// Rows of `width` elements to rows of `padded` (zeros behind them): operands
// whose rows are not 16-byte aligned.
template <typename U>
__global__ __launch_bounds__(256) void pad_kernel(const U* in, int64_t stride, U* out, int64_t rows,
                                                  int32_t width, int32_t padded) {
  const int64_t step = (int64_t)gridDim.x * 256, all = rows * padded;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t r = i / padded;
    const int32_t c = (int32_t)(i % padded);
    out[i] = c < width ? in[r * stride + c] : (U)0;
  }
}

}  // namespace ctcpb_lm
