// 8-bit codes: signed whole numbers in -127..127, or e4m3 floats (4 bits of exponent, 3 of
// fraction, up to 448).  A code stands for itself times a scale.
#pragma once
#include "common.h"

namespace ctcpb_lm {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ inline float bits_f32(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ inline uint32_t f32_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kNanBits = 0x7fc00000u;

// The scale of a block whose largest magnitude has the bits `most`: the least power of two u
// with most <= top * u, no less than 2^-126, 0 for 0, NaN where a value is not finite.
// Powers of two make what follows exact: value / u and old u / new u are, so a code is the
// nearest one to its value, whichever way it is computed, and a block whose scale grows
// is rescaled by a shift (of e4m3 codes: without loss but in the smallest ones).  For e4m3
// it costs nothing; whole numbers have on average 1.44 times the step of a scale of most/127.
// top = M 2^K with M in [1, 2): the exponent of most, less K, and one more if its fraction
// is above M's.
template <typename C>
__device__ inline uint32_t unit_bits(uint32_t most) {
  if (most >= kInfBits) return kNanBits;
  if (most == 0) return 0;
  const int e = (int)((most + (0x7fffffu - C::kTopFraction)) >> 23) - C::kTopExponent;
  return (uint32_t)(e < 1 ? 1 : e) << 23;
}

// The largest finite value of a type.
template <typename T>
constexpr float kLargest = __is_same(T, _Float16) ? 65504.0f
                           : __is_same(T, __bf16) ? 0x1.fep127f
                                                  : 0x1.fffffep127f;

// What values are multiplied by to become codes: 1 / u, or 0 for a scale that is 0 or not
// finite, whose codes are 0.
__device__ inline float inverse_unit(float u) {
  return u >= bits_f32(1u << 23) && u < bits_f32(kInfBits) ? 1.0f / u : 0.0f;
}

// The low bytes of four words.
__device__ inline uint32_t low_bytes(float a, float b, float c, float d) {
  const uint32_t lo = __builtin_amdgcn_perm(f32_bits(b), f32_bits(a), 0x0c0c0400u);
  return lo | __builtin_amdgcn_perm(f32_bits(d), f32_bits(c), 0x04000c0cu);
}

struct Int8 {
  static constexpr uint32_t kTopFraction = 0x7e0000u;   // 127 = 1.984375 * 2^6
  static constexpr int kTopExponent = 6;

  // Four numbers of at most 127.5 below 2^22, rounded to whole ones (ties to even): adding
  // 1.5 * 2^23 leaves them in the low bits.
  static __device__ uint32_t round4(float a, float b, float c, float d) {
    constexpr float M = 12582912.0f;
    return low_bytes(a + M, b + M, c + M, d + M);
  }
  static __device__ void values4(uint32_t w, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)(int32_t)(int8_t)(w >> (8 * i));
  }

  // As f16 operands of a product, codes are 1 / kUnit of themselves: a byte with its sign bit
  // turned is code + 128, as the bits of an f16 value that times 2^-24; one multiplication
  // and subtraction make the code of it, two at a time.
  static constexpr bool kNan = false;   // every code is a number
  static constexpr float kUnit = 512.0f;
  static __device__ f16x2 centred(uint32_t two) {
    const f16x2 up = {(_Float16)32768.0f, (_Float16)32768.0f};
    const f16x2 mid = {(_Float16)-0.25f, (_Float16)-0.25f};
    return __builtin_elementwise_fma(__builtin_bit_cast(f16x2, two), up, mid);
  }
  static __device__ uint32_t prepared(uint32_t w) { return w ^ 0x80808080u; }
  // codes 0, 1 or 2, 3 of a prepared word
  template <bool HIGH>
  static __device__ f16x2 two(uint32_t w) {
    return centred(__builtin_amdgcn_perm(0, w, HIGH ? 0x0c030c02u : 0x0c010c00u));
  }
  // codes J and J + 1 (J = 0 or 2) of two prepared words, each pair (a's, b's)
  template <int J>
  static __device__ void across(uint32_t a, uint32_t b, f16x2 (&to)[2]) {
    to[0] = centred(__builtin_amdgcn_perm(b, a, J ? 0x0c060c02u : 0x0c040c00u));
    to[1] = centred(__builtin_amdgcn_perm(b, a, J ? 0x0c070c03u : 0x0c050c01u));
  }
};

struct E4m3 {
  static constexpr uint32_t kTopFraction = 0x600000u;   // 448 = 1.75 * 2^8
  static constexpr int kTopExponent = 8;

  static __device__ uint32_t round4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  }
  static __device__ void values4(uint32_t w, float (&v)[4]) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    v[0] = a[0];
    v[1] = a[1];
    v[2] = b[0];
    v[3] = b[1];
  }

  static constexpr bool kNan = true;
  static constexpr float kUnit = 1.0f;
  static __device__ uint32_t prepared(uint32_t w) { return w; }
  template <bool HIGH>
  static __device__ f16x2 two(uint32_t w) {
    return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HIGH));
  }
  template <int J>
  static __device__ void across(uint32_t a, uint32_t b, f16x2 (&to)[2]) {
    const uint32_t w = __builtin_amdgcn_perm(b, a, J ? 0x07030602u : 0x05010400u);
    to[0] = two<false>(w);
    to[1] = two<true>(w);
  }
};

// N values of type T as loaded (N * sizeof(T) bytes at once), and what is asked of them.
template <typename T, int N>
struct Values {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  uint32_t w[kWords > 0 ? kWords : 1];

  __device__ void load(const void* p) {
    if constexpr (N == 1) {
      if constexpr (sizeof(T) == 2)
        w[0] = *static_cast<const uint16_t*>(p);
      else
        w[0] = *static_cast<const uint32_t*>(p);
    } else if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 x = static_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
      }
    } else {
      static_assert(kWords == 2, "values of 4, 8 or 16 k bytes");
      const u32x2 x = *static_cast<const u32x2*>(p);
      w[0] = x[0];
      w[1] = x[1];
    }
  }

  // The same from an address that is a multiple of a value's size only; `count` of them, then
  // zeros.
  __device__ void load_some(const void* p, int count) {
    if (count >= N) {
      __builtin_memcpy(w, p, sizeof(w));
      return;
    }
#pragma unroll
    for (uint32_t& x : w) x = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < count) {
        if constexpr (sizeof(T) == 2)
          w[i / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i] << (i % 2 * 16);
        else
          w[i] = static_cast<const uint32_t*>(p)[i];
      }
    }
  }

  // Raises `most`, which holds magnitudes as bits: two 16-bit ones, or one of 32.  As whole
  // numbers they order as the values do, infinities and NaN above all.
  __device__ void raise(uint32_t& most) const {
    if constexpr (sizeof(T) == 2) {
      u16x2 m = __builtin_bit_cast(u16x2, most);
#pragma unroll
      for (int i = 0; i < (kWords > 0 ? kWords : 1); ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
      most = __builtin_bit_cast(uint32_t, m);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) most = max(most, w[i] & 0x7fffffffu);
    }
  }
  // The larger of what raise() left, as the bits of a float32 value.
  static __device__ uint32_t magnitude(uint32_t most) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t m = max(most & 0xffffu, most >> 16);
      if constexpr (__is_same(T, __bf16)) return m << 16;
      return f32_bits((float)__builtin_bit_cast(_Float16, (uint16_t)m));
    }
    return most;
  }

  __device__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return bits_f32(w[i]);
    const uint32_t h = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
    if constexpr (__is_same(T, __bf16)) return bits_f32(h << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
  }
};

}  // namespace ctcpb_lm
