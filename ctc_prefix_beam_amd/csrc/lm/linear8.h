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

// What a row's largest magnitude (as bits) makes of it.
struct RowScale {
  float scale, up, unit, inverse;
  bool some;   // it has codes other than 0
  __device__ RowScale(uint32_t most) {
    const bool finite = most < kInfBits;
    scale = finite ? bits_f32(most) / 127.0f : bits_f32(kNanBits);
    // away from the subnormal numbers, where reciprocals overflow
    up = scale < 0x1p-60f ? 0x1p64f : 1.0f;
    unit = scale * up;
    some = finite && scale > 0.0f;
    inverse = some ? 1.0f / unit : 0.0f;
  }
};

// Codes of N values of a row.  1.5 * 2^23 added to a quotient leaves its nearest whole number in
// the sum's low bits, which are the code.  The reciprocal puts a quotient on the wrong side of a
// half only where it is within 2^-16 of one: then what is left of the value tells.
// ANY: `count` of them are there, and `to` may be any address.
template <typename T, int N, bool ANY>
__device__ inline void quantize_piece(const Values<T, N>& x, const RowScale& r, int8_t* to,
                                      int count) {
  constexpr float M = 12582912.0f;
  float v[N], y[N], most = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = x.at(i);
  const bool small = r.up != 1.0f;   // the same for the whole row
  if (small) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= r.up;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    y[i] = __builtin_fmaf(v[i], r.inverse, M);
    most = fmaxf(most, fabsf(__builtin_fmaf(v[i], r.inverse, M - y[i])));
  }
  if (most > 0.4999f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // what is left of v: exact where it matters, a multiple of half the unit's last bit
      const float n = y[i] - M, left = __builtin_fmaf(-n, r.unit, v[i]), half = 0.5f * r.unit;
      const bool odd = (int)n & 1;
      if (left > half || (left == half && odd))
        y[i] += 1.0f;
      else if (left < -half || (left == -half && odd))
        y[i] -= 1.0f;
    }
  }
  if (small) {   // a subnormal scale may be much less than 1/127 of the largest value
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = fminf(fmaxf(y[i], M - 127.0f), M + 127.0f);
  }
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = low_bytes(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
  if constexpr (ANY) {
    if (count >= N) {
      __builtin_memcpy(to, w, N);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < count) to[i] = (int8_t)(w[i / 4] >> (i % 4 * 8));
    }
  } else if constexpr (N == 8) {
    *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[1]};
  } else {
    *reinterpret_cast<uint32_t*>(to) = w[0];
  }
}

// Values of piece p of a row of `hidden`.
template <bool ANY, typename T, int N>
__device__ inline void load_piece(Values<T, N>& v, const char* x, int32_t p, int32_t hidden) {
  const char* at = x + (int64_t)p * (N * (int)sizeof(T));
  if constexpr (ANY)
    v.load_some(at, hidden - p * N);
  else
    v.load(at);
}

// A row's pieces lane, lane + LANES, .. : their largest magnitude, of which a caller with several
// waves to a row makes the row's.  The last kQuantHeld of them are kept for write().  ANY: rows
// begin on a value's size only, and the last piece may not be whole.
constexpr int kQuantHeld = 8;
template <typename T, int N, bool ANY, int LANES>
struct RowPieces {
  static constexpr int U = kQuantHeld;
  Values<T, N> held[U];

  __device__ uint32_t largest(const char* x, int32_t hidden, int32_t per, int lane) {
    uint32_t most = 0;
    for (int32_t p0 = 0; p0 < per; p0 += U * LANES) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t p = p0 + u * LANES + lane;
        if (p < per) {
          load_piece<ANY>(held[u], x, p, hidden);
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
    return most;
  }

  __device__ void write(const char* x, int32_t hidden, int32_t per, int lane, const RowScale& r,
                        int8_t* codes) {
    const bool again = per > U * LANES;
    for (int32_t p0 = 0; p0 < per; p0 += U * LANES)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t p = p0 + u * LANES + lane;
        if (p >= per) continue;
        if (again) load_piece<ANY>(held[u], x, p, hidden);
        if (!r.some) {
#pragma unroll
          for (uint32_t& w : held[u].w) w = 0;
        }
        quantize_piece<T, N, ANY>(held[u], r, codes + p * N, hidden - p * N);
      }
  }
};

// W waves to a row: one, and four rows to a workgroup, or four.  Bound by memory: 20000 rows of
// 4096 f16 50 to 56 us, up to 4.9 TB/s; 8192 of 2048 bf16 16 us, of which moving the 50 MB takes 10; 875 of
// 387 f32 4.7 us.  Pieces that begin anywhere (ANY): 4000 rows of 2047 bf16 14.5 us a call, 20.4
// value by value.
template <typename T, int N, bool ANY, int W>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs a) {
  constexpr int kLanes = 64 * W;
  __shared__ uint32_t part[4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  if (row >= a.rows) return;   // (of W = 4, no workgroup)
  const int lane = threadIdx.x % kLanes;
  const char* x = a.x + row * a.x_row;
  RowPieces<T, N, ANY, kLanes> pieces;
  uint32_t most = pieces.largest(x, a.hidden, a.per, lane);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) most = max(most, part[w]);
  }
  const RowScale r(most);
  if (lane == 0) a.scales[row] = r.scale;
  int8_t* codes = a.codes + row * a.codes_row;
  pieces.write(x, a.hidden, a.per, lane, r, codes);
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

// The product is that of gemm.h, with its tiles: 128 bytes of k are 128 codes.  Bound by the LDS
// that feeds the matrix units, which are busy in 50 % of the cycles: of codes, 8192 x 8192 x 2048
// bf16 120 to 127 us, up to 2300 TOP/s, and 8192^3 407 to 411, 2700 (the library's int8 product: 1740
// and 2080); 20000 x 1024 x 4096 83 us, 2020. One wave to a SIMD with a tile of 128 x 128, which reads a third less from
// LDS, took 2.3 times as long.
//
// What follows a sum: scales and bias, in float32.  Every kernel rounds alike (no product is
// contracted with the sum but the last, by a power of two), so that a row's results do not
// depend on how many rows there are.
__device__ inline float finish(int32_t sum, const TwoFactors& x, float w, float bias) {
#pragma clang fp contract(off)
  float y = __builtin_fmaf((float)sum * x.first * w, x.second, bias);
  asm("" : "+v"(y));   // a float32 value: else f16 results may be rounded from the exact sum
  return y;
}

// WIDE: rows of out begin on 16 bytes and have whole pieces of them.
template <typename T, bool WIDE>
struct Linear8Epilogue {
  T* out;
  int64_t ld;
  const float *w_scale, *bias, *x_scale;   // bias: or null
  int32_t* planes;     // parts of k: [part][n][pitch], or null
  int32_t pitch;       // of m in a plane, a multiple of 4
  int32_t M, N;

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
    // kWide channels of 16 rows, which lie in different banks and begin where four values can be
    // stored at once.  Of f32 half as many, so that as many workgroups share a CU as without.
    typedef T T4 __attribute__((ext_vector_type(4)));
    constexpr int kHalves = sizeof(T) == 2 ? 2 : 1, kWide = kHalves * 16, kPitch = kWide + 4;
    static_assert(kPitch * sizeof(T) % sizeof(T4) == 0, "rows begin between two stores");
    __shared__ __align__(16) T stage[WIDE ? 1 : WM * WN][WIDE ? 1 : 16 * kPitch];
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
#pragma unroll
          for (int r = 0; r < 4; ++r) y[h][r] = finish(acc[i + h][j][r], sx, sw[h][r], b[h][r]);
        T* to = out + n * ld;
        const int m = mb + i * 16;
        if constexpr (sizeof(T) == 2 && WIDE) {
          const TilePair<T> t(y[0], y[1]);
          const int at = m + TilePair<T>::at(g);
          if (n < N && at < M) t.store(to + at);
        } else if constexpr (WIDE) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (n < N && m + h * 16 + g * 4 < M)
              *reinterpret_cast<f32x4*>(to + m + h * 16 + g * 4) = y[h];
        } else {
          // Rows that begin anywhere: the tile goes through LDS, so that a store has neighbouring
          // values of a few rows, not a few of many (8192 x 8191 x 2048 bf16 169 us a call, 222
          // without)
          T* at = stage[wm * WN + wn];
          const int first = n - c;   // of the tile's 16 rows
#pragma unroll
          for (int part = 0; part < 2; part += kHalves) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              T4 v;
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] = (T)y[part + h][r];
              *reinterpret_cast<T4*>(at + c * kPitch + h * 16 + g * 4) = v;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < kWide / 4; ++q) {
              const int row = (q * 64 + lane) / kWide, mm = lane % kWide;
              const T v = at[row * kPitch + mm];
              const int ch = m + part * 16 + mm;
              if (first + row < N && ch < M) out[(int64_t)(first + row) * ld + ch] = v;
            }
            __builtin_amdgcn_wave_barrier();
          }
        }
      }
    }
  }
};

// Adds the planes of parts of k (whole numbers: in any order) and finishes the result.
template <typename T>
__global__ __launch_bounds__(256) void linear8_join_kernel(Linear8Epilogue<T, false> ep,
                                                           int32_t parts) {
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
            (T)finish(sum[r], sx, ep.w_scale[m + r], ep.bias ? ep.bias[m + r] : 0.0f);
  }
}

// ---------------------------------------------------------- few rows ----
//
// Up to 16 * NT rows of x against all of w, in one launch: what it cannot do without is reading w
// once, and for small layers a launch.  A workgroup of 16 waves to a CU takes the codes of x into
// LDS, and quantises them for itself from up to kFewValues values (which costs less than a launch
// of its own).  Then KW waves share the k of a tile of 16 channels, 16 / KW tiles at a time; the
// next tiles' first weights are on their way while the waves' sums are added.  Weights go from
// memory straight into the registers of the matrix instruction, kFewHeld of them a lane at a
// time.  On the GPU, with weights that its caches hold: 32 rows x 5000 channels of 512, bf16, 8.1
// us; a row of codes with 8192 channels of 2048 (16.8 MB) 5.7.  Long rows are quantised by several
// waves each: a row of 4096 with 4096 channels 6.4 us (8.3 with a launch for that), of 16384 17.5
// (24.9).
constexpr int32_t kFewValues = 16384;
constexpr int32_t kFewCodes = 124 * 1024;   // of a CU's 160 KB of LDS; the waves' sums take 32 KB
constexpr int kFewHeld = 8;

struct FewArgs {
  const char* x;
  int64_t x_row;           // bytes
  const float *x_scale;    // of codes, else null
  const int8_t* w;
  int64_t w_row;
  const float *w_scale, *bias;
  char* out;
  int64_t out_row;         // elements
  int32_t rows, hidden, features;
  int32_t padded;          // bytes of a row of w that can be read
  int32_t per;             // pieces of a row of x
  int32_t ways_log;        // 2^this waves quantise a row: as many of the 16 as it has pieces for
};

// Codes and scales of the rows, up to 16 * R: a wave has a part of row `wave >> ways_log`, or (R =
// 2) rows `wave` and wave + 16, whose loads and reductions overlap.  P pieces a lane to each.
// `most_of`: room for 16 waves' maxima.
template <typename X, int N, bool ANY, int P, int R>
__device__ inline void quantize_few(const FewArgs& a, int wave, int lane, int8_t* codes, int pitch,
                                    float* sx, uint32_t* most_of) {
  const int ways = R == 1 ? 1 << a.ways_log : 1, n0 = R == 1 ? wave >> a.ways_log : wave;
  const int first = (wave & (ways - 1)) * 64 + lane, step = 64 * ways;   // of the lane's pieces
  Values<X, N> held[R][P];
  uint32_t most[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = min(n0 + r * 16, a.rows - 1);   // (the last row again: not kept)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (first + p * step < a.per) {
        load_piece<ANY>(held[r][p], a.x + n * a.x_row, first + p * step, a.hidden);
      } else {
#pragma unroll
        for (uint32_t& w : held[r][p].w) w = 0;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    most[r] = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) held[r][p].raise(most[r]);
    most[r] = Values<X, N>::magnitude(most[r]);
  }
  for (int s = 1; s < 64; s <<= 1)
#pragma unroll
    for (int r = 0; r < R; ++r) most[r] = max(most[r], (uint32_t)__shfl_xor((int)most[r], s));
  if (R == 1 && ways > 1) {
    if (lane == 0) most_of[wave] = most[0];
    __syncthreads();
    for (int w = 0; w < ways; ++w) most[0] = max(most[0], most_of[(wave & -ways) + w]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = n0 + r * 16;
    const RowScale q(most[r]);
    if (n < a.rows) {
      if (first == 0) sx[n] = q.scale;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int k = (first + p * step) * N;
        if (!q.some) {
#pragma unroll
          for (uint32_t& w : held[r][p].w) w = 0;
        }
        if (first + p * step < a.per)
          quantize_piece<X, N, ANY>(held[r][p], q, codes + n * pitch + k, a.hidden - k);
      }
    }
  }
}

// X: type of x (int8_t: codes), of which a piece of N is 16 bytes; KW: 4, or 16 for few channels.
template <typename T, typename X, bool ANY, int NT, int KW>
__global__ __launch_bounds__(1024) void linear8_few_kernel(FewArgs a) {
  constexpr int U = kFewHeld, G = 16 / KW, N = 16 / (int)sizeof(X);
  extern __shared__ __align__(16) char few_lds[];
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % KW, mine = wave / KW;   // of a tile's k, and of the G tiles
  const int steps = (a.padded + 63) / 64;
  const int pitch = steps * 64 + 16;   // rows begin in different banks
  int8_t* codes = reinterpret_cast<int8_t*>(few_lds);
  i32x4* parts = reinterpret_cast<i32x4*>(few_lds + a.rows * pitch);   // [wave][NT][lane]
  float* sx = reinterpret_cast<float*>(parts + 16 * NT * 64);
  const int tiles = (a.features + 15) / 16;
  u32x4 held[U];
  // the lane's weights of U steps of a tile from step s on, every KW-th one
  const auto load = [&](int tile, int s) {
    const int8_t* row = a.w + (int64_t)min(tile * 16 + c, a.features - 1) * a.w_row;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + KW * u) * 64 + g * 16;
      held[u] = u32x4{0, 0, 0, 0};
      if (k < a.padded) held[u] = *reinterpret_cast<const u32x4*>(row + k);
    }
  };
  int first = blockIdx.x * G;   // of the G tiles
  load(first + mine, part);
  if constexpr (sizeof(X) == 1) {
    for (int n = wave; n < a.rows; n += 16) {
      const char* x = a.x + n * a.x_row;
#pragma unroll 4
      for (int p = lane; p < a.per; p += 64) {
        int8_t* to = codes + n * pitch + p * N;
        if constexpr (ANY) {
          if (a.hidden - p * N >= N)
            __builtin_memcpy(to, x + p * N, N);
          else
            for (int k = p * N; k < a.hidden; ++k) codes[n * pitch + k] = (int8_t)x[k];
        } else {
          *reinterpret_cast<u32x4*>(to) = reinterpret_cast<const u32x4*>(x)[p];
        }
      }
      if (lane == 0) sx[n] = a.x_scale[n];
    }
  } else {
    // Pieces a lane, if there is more than one: rows * hidden is at most kFewValues, and more than 8
    // waves have a part, so up to 32 / N of them
    static_assert(kFewValues <= 16384, "more pieces than that");
    uint32_t* most_of = reinterpret_cast<uint32_t*>(parts);
    const int lanes = NT == 1 ? 64 << a.ways_log : 64;
    if (a.per <= lanes)
      quantize_few<X, N, ANY, 1, NT>(a, wave, lane, codes, pitch, sx, most_of);
    else if (a.per <= 2 * lanes)
      quantize_few<X, N, ANY, 2, NT>(a, wave, lane, codes, pitch, sx, most_of);
    else if (N == 8 || a.per <= 4 * lanes)
      quantize_few<X, N, ANY, 4, NT>(a, wave, lane, codes, pitch, sx, most_of);
    else
      quantize_few<X, N, ANY, N == 4 && NT == 1 ? 8 : 4, NT>(a, wave, lane, codes, pitch, sx,
                                                             most_of);
  }
  for (int n = wave; n < a.rows; n += 16)
    for (int k = a.hidden + lane; k < steps * 64; k += 64) codes[n * pitch + k] = 0;
  __syncthreads();
  for (; first < tiles; first += gridDim.x * G) {
    i32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    for (int s = part;; s += KW * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s + KW * u < steps) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            // rows past the last one repeat it, and are not kept
            const int n = min(t * 16 + c, a.rows - 1);
            const i32x4 xf = *reinterpret_cast<const i32x4*>(codes + n * pitch +
                                                             (s + KW * u) * 64 + g * 16);
            acc[t] = Frag<int8_t>::mac(__builtin_bit_cast(i32x4, held[u]), xf, acc[t]);
          }
        }
      }
      if (s + KW * U >= steps) break;
      load(first + mine, s + KW * U);
    }
    if (first + (int)gridDim.x * G < tiles) load(first + gridDim.x * G + mine, part);
    __syncthreads();   // the tiles before have been added
#pragma unroll
    for (int t = 0; t < NT; ++t) parts[(wave * NT + t) * 64 + lane] = acc[t];
    __syncthreads();
    // a thread has a channel and a row of x: 16 * G channels, of which 16 to a tile, next to
    // each other in out
    for (int i = threadIdx.x; i < 256 * NT * G; i += 1024) {
      const int m = i % (16 * G), n = i / (16 * G);
      const int64_t at = (int64_t)first * 16 + m;
      if (n >= a.rows || at >= a.features) continue;
      int32_t sum = 0;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const i32x4* from = parts + ((m / 16 * KW + w) * NT + (n >> 4)) * 64;
        sum += reinterpret_cast<const int32_t*>(from + ((m & 15) >> 2) * 16 + (n & 15))[m & 3];
      }
      reinterpret_cast<T*>(a.out)[n * a.out_row + at] =
          (T)finish(sum, TwoFactors(sx[n]), a.w_scale[at], a.bias ? a.bias[at] : 0.0f);
    }
  }
}

}  // namespace ctcpb_lm
