// Products of 8-bit rows: out[n, m] = (sum_k x[n, k] w[m, k]) sx[n] sw[m] + bias[m], with whole
// codes and a scale for each row of x (a token) and of w (a channel).  The sum is exact in 32
// bits, so no way of cutting it up changes the result, and what it loses against the product
// of the values is the codes' rounding alone.
#pragma once
#include "codes.h"
#include "gemm.h"

namespace ctcpb_lm {

// -------------------------------------------------------------- quantise --
//
// scale = max |x| / 127 of a row, as a float32 number; code = x / scale rounded to the nearest
// whole number, ties to the even one, of the exact quotient: x times the reciprocal is only
// looked at again where it lies next to a half.  A row with a value that is not finite has
// the scale NaN and codes of 0, so that what is made of it is NaN.
struct QuantArgs {
  const char* x;
  int64_t x_row;          // bytes
  int8_t* codes;
  int64_t codes_row;
  float* scales;
  int32_t rows, hidden;
  int32_t padded;         // codes from `hidden` to here are zeros
  int32_t per;            // pieces of a row
};

// Codes of N values: times `up` (a power of two), then over `unit`.
template <typename T, int N>
__device__ inline void quantize_piece(const Values<T, N>& x, float up, float unit, float inverse,
                                      int8_t* to) {
  constexpr float M = 12582912.0f;   // 1.5 * 2^23: sums with it are whole
  float v[N], n[N];
  bool near = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = x.at(i) * up;
    n[i] = __builtin_fmaf(v[i], inverse, M) - M;
    near = near || fabsf(__builtin_fmaf(v[i], inverse, -n[i])) > 0.4999f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // what is left of v: exact where it matters, a multiple of half the unit's last bit
      const float left = __builtin_fmaf(-n[i], unit, v[i]), half = 0.5f * unit;
      const bool odd = (int)n[i] & 1;
      if (left > half || (left == half && odd))
        n[i] += 1.0f;
      else if (left < -half || (left == -half && odd))
        n[i] -= 1.0f;
    }
  }
  uint32_t w[N > 4 ? N / 4 : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) n[i] = fminf(fmaxf(n[i], -127.0f), 127.0f);
  if constexpr (N == 1) {
    *to = (int8_t)(int)n[0];
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = Int8::round4(n[4 * i], n[4 * i + 1], n[4 * i + 2], n[4 * i + 3]);
    if constexpr (N == 8)
      *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
    else
      *reinterpret_cast<uint32_t*>(to) = w[0];
  }
}

// W waves to a row: one, and four rows to a workgroup, or four.  Bound by memory.
constexpr int kQuantHeld = 8;   // pieces a lane keeps between the two passes
template <typename T, int N, int W>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs a) {
  constexpr int U = kQuantHeld, kLanes = 64 * W;
  __shared__ uint32_t part[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  if (row >= a.rows) return;   // (of W = 4, no workgroup)
  const int lane = threadIdx.x % kLanes;
  const char* x = a.x + row * a.x_row;
  Values<T, N> held[U];
  uint32_t most = 0;
  for (int32_t p0 = 0; p0 < a.per; p0 += U * kLanes) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t p = p0 + u * kLanes + lane;
      if (p < a.per) {
        held[u].load(x + (int64_t)p * (N * (int)sizeof(T)));
      } else {
#pragma unroll
        for (uint32_t& w : held[u].w) w = 0;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) held[u].raise(most);
  }
  most = Values<T, N>::magnitude(most);
  for (int s = 1; s < 64; s <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, s));
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) most = max(most, part[w]);
  }
  const bool finite = most < kInfBits;
  const float scale = finite ? bits_f32(most) / 127.0f : bits_f32(kNanBits);
  if (lane == 0) a.scales[row] = scale;
  // away from the subnormal numbers, where reciprocals overflow
  const float up = scale < 0x1p-60f ? 0x1p64f : 1.0f;
  const float unit = scale * up;
  const bool some = finite && scale > 0.0f;
  const float inverse = some ? 1.0f / unit : 0.0f;
  int8_t* codes = a.codes + row * a.codes_row;
  const bool again = a.per > U * kLanes;
  for (int32_t p0 = 0; p0 < a.per; p0 += U * kLanes)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t p = p0 + u * kLanes + lane;
      if (p >= a.per) continue;
      if (again) held[u].load(x + (int64_t)p * (N * (int)sizeof(T)));
      if (!some) {
#pragma unroll
        for (uint32_t& w : held[u].w) w = 0;
      }
      quantize_piece<T, N>(held[u], up, unit, inverse, codes + p * N);
    }
  for (int32_t k = a.hidden + lane; k < a.padded; k += kLanes) codes[k] = 0;
}

// --------------------------------------------------------------- product --

// A scale of x in two factors, the second 1 but for scales so large that a sum times them
// could pass the end of float32 before the other scale takes it back.
struct TwoFactors {
  float first, second;
  __device__ TwoFactors(float s) : first(s > 0x1p64f ? s * 0x1p-64f : s),
                                   second(s > 0x1p64f ? 0x1p64f : 1.0f) {}
};

// What follows the sums: scales and bias, in float32, and one rounding.
template <typename T>
struct Linear8Epilogue {
  T* out;
  int64_t ld;
  const float *w_scale, *bias, *x_scale;   // bias: or null
  int32_t* planes;     // parts of k: [part][n][pitch], or null
  int32_t pitch;       // of m in a plane, a multiple of 4
  int32_t M, N;
  bool wide;           // rows of out can be written 16 bytes at a time

  static constexpr bool kJoins = false;
  template <int BM, int BN>
  static constexpr int wanted() {
    return 2 * BM + BN;
  }
  template <int BM, int BN, int W>
  __device__ void fetch(const Place& at, float* to, int wave, int lane) const {
    const int m = at.m * BM;
    fetch_floats<BM, W>(w_scale + m, M - m, to, 0, wave, lane);
    fetch_floats<BM, W>(bias ? bias + m : w_scale, bias ? M - m : 0, to + BM, BM / 64, wave, lane);
    fetch_floats<BN, W>(x_scale + at.n0, N - at.n0, to + 2 * BM, 2 * BM / 64, wave, lane);
  }

  template <int TM, int TN, int WM, int WN>
  __device__ void run(i32x4 (&acc)[TM][TN], const Place& at, int wm, int wn, int lane, float2*,
                      const float* got) {
    constexpr int BM = WM * TM * 16;
    const int g = lane >> 4, c = lane & 15;
    const int mb = (at.m * WM + wm) * TM * 16;
    if (planes) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = at.n0 + (wn * TN + j) * 16 + c;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int m = mb + i * 16 + g * 4;
          if (n < N && m < M)
            *reinterpret_cast<i32x4*>(planes + ((int64_t)at.split * N + n) * pitch + m) = acc[i][j];
        }
      }
      return;
    }
    const float* mine = got + wm * TM * 16 + g * 4;
#pragma unroll
    for (int i = 0; i < TM; i += 2) {
      f32x4 sw[2], b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sw[h] = *reinterpret_cast<const f32x4*>(mine + (i + h) * 16);
        b[h] = *reinterpret_cast<const f32x4*>(mine + BM + (i + h) * 16);
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int k = (wn * TN + j) * 16 + c, n = at.n0 + k;
        const TwoFactors sx(got[2 * BM + k]);
        f32x4 y[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          y[h] = __builtin_convertvector(acc[i + h][j], f32x4) * sx.first * sw[h] * sx.second + b[h];
        T* to = out + n * ld;
        if (sizeof(T) == 2 && wide) {
          if constexpr (sizeof(T) == 2) {
            const TilePair<T> t(y[0], y[1]);
            const int m = mb + i * 16 + TilePair<T>::at(g);
            if (n < N && m < M) t.store(to + m);
          }
          continue;
        }
        if (n >= N) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = mb + (i + h) * 16 + g * 4;
          if (sizeof(T) == 4 && wide) {
            if (m < M) *reinterpret_cast<f32x4*>(to + m) = y[h];
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (m + r < M) to[m + r] = (T)y[h][r];
          }
        }
      }
    }
  }
};

// Adds the planes of parts of k (whole numbers: in any order) and finishes the result.
template <typename T>
__global__ __launch_bounds__(256) void linear8_join_kernel(Linear8Epilogue<T> ep, int32_t parts) {
  const int32_t quads = ep.pitch / 4;
  const int64_t step = (int64_t)gridDim.x * 256, all = (int64_t)ep.N * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += step) {
    const int64_t n = i / quads;
    const int32_t m = (int32_t)(i % quads) * 4;
    i32x4 sum = {0, 0, 0, 0};
#pragma unroll 4
    for (int p = 0; p < parts; ++p)
      sum += *reinterpret_cast<const i32x4*>(ep.planes + ((int64_t)p * ep.N + n) * ep.pitch + m);
    const TwoFactors sx(ep.x_scale[n]);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (m + r < ep.M)
        ep.out[n * ep.ld + m + r] =
            (T)((float)sum[r] * sx.first * ep.w_scale[m + r] * sx.second +
                (ep.bias ? ep.bias[m + r] : 0.0f));
  }
}

}  // namespace ctcpb_lm
