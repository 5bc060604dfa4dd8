// Types and wave helpers shared by the language-model operators.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace ctcpb_lm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ inline float neg_inf() { return -__builtin_huge_valf(); }
__device__ inline float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// exp(x) for x <= 0: 2^(x log2 e) is off by |x| 2^-24, below what 16-bit outputs
// show; f32 takes the library's exponential.
template <typename T>
__device__ inline float exp_of(float x) {
  if constexpr (sizeof(T) == 4) return expf(x);
  return exp_fast(x);
}

// Maximum / sum over the four lanes l, l^16, l^32, l^48.
__device__ inline float max_over_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ inline float sum_over_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// A paged cache of keys or values.
struct CacheView {
  char* data;
  int64_t page, token, head;   // strides in bytes
};

}  // namespace ctcpb_lm
