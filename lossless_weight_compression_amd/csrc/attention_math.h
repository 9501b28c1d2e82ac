// attention_math.h -- what the attention kernels share: matrix products of the
// 16-bit types, exponentials, and exchanges between the lanes that hold a query
// row (device code only).
#pragma once
#include "step_common.h"

namespace enc {
namespace {

constexpr float kLowest = -3.402823466e38f;   // finite: differences with it are not NaN
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kSlack2 = 8.0f, kSlack = kSlack2 * kLn2;

// e^x. Scores stay in natural units until here: the difference of two finite
// scores does not overflow, a score times log2(e) may.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
template <typename T> struct Half;
template <> struct Half<__bf16> {
  static constexpr uint32_t kExp = 0x7F80u;
  static constexpr float kLift2 = 0.f, kLift = 0.f;
  static __device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};
template <> struct Half<_Float16> {
  static constexpr uint32_t kExp = 0x7C00u;
  // P is held 2^6 larger (at most 2^14): FP16 loses precision below 2^-14, and
  // many keys of little weight together still count
  static constexpr float kLift2 = 6.f, kLift = kLift2 * kLn2;
  static __device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
};

// Maximum / sum over the four lanes that hold the same query row (l, l ^ 16,
// l ^ 32, l ^ 48), by exchanging rows of 16 lanes: no LDS round trip.
__device__ __forceinline__ float rows_max(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float rows_sum(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 read_transposed(const void *lds) {
  typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(uintptr_t)lds));
}

}  // namespace
}  // namespace enc
