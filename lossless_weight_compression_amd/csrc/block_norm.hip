// block_norm.hip -- the norm after a block, its gate, the residual sum and the
// norm before the next block in one pass over the rows (enc_block_norm).
//
//   z = y rsqrt(mean(y^2) + eps) w_post,  h' = a h + s g z,
//   x = h' rsqrt(mean(h'^2) + eps) w_pre
//
// Every value is read once, held in fp32 and rounded once; x is taken from h'
// as it was before rounding. The bound is HBM traffic (about 9 flops a value);
// for a few rows it is the time from the first load to the last store. So a row
// is one workgroup's, all of it in registers, 8 consecutive values to a thread
// and NV times that: all of a row's loads (weights and gates too) are on their
// way before the first sum, and a row costs one barrier, or two with the norm
// after the block. Above 16384 values (NV = 4) weights and gates are loaded when
// they are needed, and still some 40 of a thread's registers spill to memory.
//
// A row's 16-byte results are stored past the caches: many rows at once come to
// 6.2 TB/s instead of 5.5, and a kernel that reads them next is no slower (two
// calls, the second on the first one's results: 155 us against 171 for 8192 rows
// of 4096, 11.8 against 14.0 for 792 of 2560).
//
// Measured: 1 row of 4096 3.4 us (a launch alone takes about 2), 792 rows of 2560
// 6.0 us, 8192 rows of 4096 (FP32 y and h, 470 MB) 76 us = 6.2 TB/s, where a
// large copy reaches 5.1; 515 odd rows of 1537, one value a load, 6.9 us. The widest
// rows (FP32 y and h, both norms): 2048 of 16384 90 us = 5.2 TB/s, 2048 of 16392 159 =
// 3.0, 1024 of 32768 134 = 3.5, one of them 14.4, 1024 of 32767 156 = 3.0.
#include "step_common.h"

#include <algorithm>

namespace enc {
namespace {

constexpr uint32_t kMaxThreads = 1024;

// Eight values of a thread as they lie in memory: two 16-byte loads of fp32, one
// of a 16-bit type, or, where rows are not aligned, one load for each value.
struct Raw {
  uint32_t w[8];
};

template <bool VEC>
__device__ __forceinline__ void load_raw(Raw &r, const void *row, uint32_t dtype, uint32_t at, uint32_t step, uint32_t n) {
#pragma unroll
  for (int e = 0; e < 8; ++e) r.w[e] = 0;
  if constexpr (VEC) {
    if (at >= n) return;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + (dtype == 3 ? 2 * at : at));
    const uint4 a = p[0];
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    if (dtype == 3) {
      const uint4 b = p[1];
      r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
    }
  } else if (dtype == 3) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e * step < n) r.w[e] = static_cast<const uint32_t *>(row)[at + e * step];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e * step < n) r.w[e] = static_cast<const uint16_t *>(row)[at + e * step];
  }
}

template <bool VEC> __device__ __forceinline__ void values_of(const Raw &r, uint32_t dtype, float (&x)[8]) {
  if (dtype == 3) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r.w[e]);
  } else if (dtype == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = VEC ? half_of<__bf16>(r.w[e >> 1], e & 1) : half_of<__bf16>(r.w[e], 0);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = VEC ? half_of<_Float16>(r.w[e >> 1], e & 1) : half_of<_Float16>(r.w[e], 0);
  }
}

template <bool VEC>
__device__ __forceinline__ void store_values(void *row, uint32_t dtype, const float (&x)[8], uint32_t at, uint32_t step,
                                             uint32_t n) {
  if constexpr (VEC) {
    if (at >= n) return;
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + (dtype == 3 ? 2 * at : at));
    if (dtype == 3) {
      store_nt16(p, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
      store_nt16(p + 1, make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])));
    } else if (dtype == 1) {
      store_nt16(p, make_uint4(pack2<__bf16>(x[0], x[1]), pack2<__bf16>(x[2], x[3]), pack2<__bf16>(x[4], x[5]),
                               pack2<__bf16>(x[6], x[7])));
    } else {
      store_nt16(p, make_uint4(pack2<_Float16>(x[0], x[1]), pack2<_Float16>(x[2], x[3]), pack2<_Float16>(x[4], x[5]),
                               pack2<_Float16>(x[6], x[7])));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t i = at + e * step;
      if (i >= n) continue;
      if (dtype == 3)
        static_cast<float *>(row)[i] = x[e];
      else
        static_cast<uint16_t *>(row)[i] = (uint16_t)(dtype == 1 ? pack2<__bf16>(x[e], 0.f) : pack2<_Float16>(x[e], 0.f));
    }
  }
}

// Sum over the 64 lanes, in every lane: quads, half rows and rows of 16 lanes by
// operand permutes, then rows exchanged. No LDS.
__device__ __forceinline__ float wave_sum(float x) {
  const auto add = [](float v, int moved) { return v + __int_as_float(moved); };
  x = add(x, __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, false));
  x = add(x, __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, false));
  x = add(x, __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, false));
  x = add(x, __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xF, 0xF, false));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the workgroup, in every thread; `side` is used once.
__device__ __forceinline__ float group_sum(float x, float *side) {
  x = wave_sum(x);
  const uint32_t waves = blockDim.x / 64;
  if (waves == 1) return x;
  if ((threadIdx.x & 63) == 0) side[threadIdx.x >> 6] = x;
  __syncthreads();
  float total = 0.f;
  for (uint32_t w = 0; w < waves; ++w) total += side[w];
  return total;
}

template <uint32_t NV, bool VEC>
__global__ __launch_bounds__(kMaxThreads) void k_block_norm(BlockNormKernelArgs k) {
  const enc_block_norm_args &a = k.a;
  __shared__ float sides[2][kMaxThreads / 64];
  const uint32_t n = a.width, threads = blockDim.x, token = k.token0 + blockIdx.x;
  // value e of chunk j: 8 consecutive ones, or, one load at a time, `threads` apart
  const uint32_t step = VEC ? 1 : threads;
  uint32_t at[NV];
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) at[j] = VEC ? (j * threads + threadIdx.x) * 8 : j * 8 * threads + threadIdx.x;
  const auto row_of = [](const void *p, uint32_t dtype, uint64_t offset) {
    return static_cast<const void *>(static_cast<const uint8_t *>(p) + offset * (dtype == 3 ? 4 : 2));
  };

  const bool post = a.flags & ENC_BLOCK_POST_NORM, offset = a.flags & ENC_BLOCK_UNIT_OFFSET;
  Raw y[NV], h[NV], g[NV], wq[NV], wp[NV];
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) {
    if (a.d_y) load_raw<VEC>(y[j], row_of(a.d_y, a.y_dtype, token * a.y_token), a.y_dtype, at[j], step, n);
    load_raw<VEC>(h[j], row_of(a.d_h, a.h_dtype, token * a.h_token), a.h_dtype, at[j], step, n);
  }
  const void *gates = a.d_gate ? row_of(a.d_gate, a.g_dtype, k.gate.quot(token) * a.gate_row) : nullptr;
  const auto load_rest = [&](uint32_t j) {
    if (a.d_gate) load_raw<VEC>(g[j], gates, a.g_dtype, at[j], step, n);
    if (a.d_w_post) load_raw<VEC>(wq[j], a.d_w_post, a.w_dtype, at[j], step, n);
    if (a.d_w_pre) load_raw<VEC>(wp[j], a.d_w_pre, a.w_dtype, at[j], step, n);
  };
  constexpr bool kEarly = NV <= 2;   // registers for them before the first sum
  if constexpr (kEarly)
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) load_rest(j);

  float x[NV][8];
  if (a.d_y) {
    float scale = a.y_scale;
    if (post) {
      float ss = 0.f;
#pragma unroll
      for (uint32_t j = 0; j < NV; ++j) {
        values_of<VEC>(y[j], a.y_dtype, x[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[j][e], x[j][e], ss);
      }
      scale = 1.0f / sqrtf(group_sum(ss, sides[0]) / (float)n + a.eps);
    }
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      if constexpr (!kEarly) load_rest(j);
      values_of<VEC>(y[j], a.y_dtype, x[j]);
      float v[8];
      if (post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= scale;
        if (a.d_w_post) {
          values_of<VEC>(wq[j], a.w_dtype, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[j][e] *= offset ? 1.f + v[e] : v[e];
        }
      }
      if (a.d_gate) {
        values_of<VEC>(g[j], a.g_dtype, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] *= v[e];
      }
      values_of<VEC>(h[j], a.h_dtype, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = fmaf(a.h_scale, v[e], a.y_scale * x[j][e]);
    }
  } else {
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      if constexpr (!kEarly) load_rest(j);
      values_of<VEC>(h[j], a.h_dtype, x[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] *= a.h_scale;
    }
  }
  if (a.d_h_out) {
    void *dst = static_cast<uint8_t *>(a.d_h_out) + token * a.h_out_token * (a.h_dtype == 3 ? 4 : 2);
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) store_values<VEC>(dst, a.h_dtype, x[j], at[j], step, n);
  }
  if (!a.d_out) return;
  float ss = 0.f;
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (VEC || at[j] + e * step < n) ss = fmaf(x[j][e], x[j][e], ss);
  const float scale = 1.0f / sqrtf(group_sum(ss, sides[1]) / (float)n + a.eps);
  void *dst = static_cast<uint8_t *>(a.d_out) + token * a.out_token * (a.out_dtype == 3 ? 4 : 2);
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[j][e] *= scale;
    if (a.d_w_pre) {
      float v[8];
      values_of<VEC>(wp[j], a.w_dtype, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] *= offset ? 1.f + v[e] : v[e];
    }
    store_values<VEC>(dst, a.out_dtype, x[j], at[j], step, n);
  }
}

template <uint32_t NV>
void launch_rows(BlockNormKernelArgs k, hipStream_t s) {
  const uint32_t chunks = (k.a.width + 8 * NV - 1) / (8 * NV), threads = (chunks + 63) / 64 * 64;
  const uint32_t most = 1u << 21;   // a grid holds fewer than 2^32 threads
  for (uint64_t token0 = 0; token0 < k.a.tokens; token0 += most) {
    k.token0 = (uint32_t)token0;
    const dim3 grid(std::min(most, k.a.tokens - k.token0)), block(threads);
    if (k.vec)
      hipLaunchKernelGGL((k_block_norm<NV, true>), grid, block, 0, s, k);
    else
      hipLaunchKernelGGL((k_block_norm<NV, false>), grid, block, 0, s, k);
  }
}

}  // namespace

hipError_t launch_block_norm(const BlockNormKernelArgs &k, hipStream_t s) {
  const uint32_t chunks = (k.a.width + 7) / 8;
  // As few values a thread as a workgroup's 1024 threads allow: two chunks to a
  // thread took 99 us for 8192 rows of 4096 against 86 with one, four 148.
  if (chunks > 2 * kMaxThreads)
    launch_rows<4>(k, s);
  else if (chunks > kMaxThreads)
    launch_rows<2>(k, s);
  else
    launch_rows<1>(k, s);
  return hipGetLastError();
}

}  // namespace enc
