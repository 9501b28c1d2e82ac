// qk_rope.hip -- norms of query and key heads, rotary embedding and type
// conversion in one pass (enc_qk_norm_rope).
//
// y = x rsqrt(mean(x^2) + eps) w over a head, then the first rot_dim values
// turned pairwise by the token's angles. Every value is read once, held in
// fp32 and rounded once. The bound is HBM traffic (about 8 flops per value):
// a head of D values is held by D/8 lanes (rounded up to a power of two, so
// its sum is a butterfly inside one wave), 8 consecutive values each, which
// makes every load and store 16 bytes or more per lane. Values are exchanged
// between the two halves of a head through LDS, written as the lane holds
// them. The table row of a token is read by all its heads from cache.
#include "step_common.h"

namespace enc {
namespace {

constexpr uint32_t kBlock = 256;

template <typename T> struct Eight;
template <> struct Eight<float> {
  static __device__ __forceinline__ void load(const void *p, float (&x)[8]) {
    const f32x4 a = static_cast<const f32x4 *>(p)[0], b = static_cast<const f32x4 *>(p)[1];
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  }
  static __device__ __forceinline__ void store(void *p, const float (&x)[8]) {
    static_cast<f32x4 *>(p)[0] = f32x4{x[0], x[1], x[2], x[3]};
    static_cast<f32x4 *>(p)[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
};
template <typename T> struct Eight16 {
  static __device__ __forceinline__ void load(const void *p, float (&x)[8]) {
    const uint4 v = *static_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < 8; ++i) x[i] = half_of<T>(w[i >> 1], i & 1);
  }
  static __device__ __forceinline__ void store(void *p, const float (&x)[8]) {
    *static_cast<uint4 *>(p) = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]),
                                          pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
  }
};
template <> struct Eight<__bf16> : Eight16<__bf16> {};
template <> struct Eight<_Float16> : Eight16<_Float16> {};

__device__ __forceinline__ void load_weight(const void *w, uint32_t dtype, uint32_t d0, float (&x)[8]) {
  if (dtype == 1)
    Eight<__bf16>::load(static_cast<const uint16_t *>(w) + d0, x);
  else if (dtype == 2)
    Eight<_Float16>::load(static_cast<const uint16_t *>(w) + d0, x);
  else
    Eight<float>::load(static_cast<const float *>(w) + d0, x);
}

template <typename TI, typename TO, uint32_t LANES>
__global__ __launch_bounds__(kBlock) void k_qk_norm_rope(QkKernelArgs k) {
  const enc_qk_args &a = k.a;
  __shared__ __align__(16) float xs[kBlock * 8];
  const uint32_t chunk = threadIdx.x % LANES, d0 = chunk * 8;
  const uint32_t item = blockIdx.x * (kBlock / LANES) + threadIdx.x / LANES;
  const bool live = item < k.items && d0 < a.head_dim;
  const uint32_t it = item < k.items ? item : k.items - 1;
  const uint32_t token = k.per_token.quot(it), head = it - token * k.per_token.d;
  const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.kv_heads;
  const uint32_t h = is_q ? head : is_v ? head - a.q_heads - a.kv_heads : head - a.q_heads;
  const uint64_t in = is_q   ? token * a.q_token + h * a.q_head
                      : is_v ? token * a.v_token + h * a.v_head
                             : token * a.k_token + h * a.k_head;
  const uint64_t out = is_q   ? token * a.q_out_token + h * a.q_out_head
                       : is_v ? token * a.v_out_token + h * a.v_out_head
                              : token * a.k_out_token + h * a.k_out_head;
  const TI *src = static_cast<const TI *>(is_q ? a.d_q : is_v ? a.d_v : a.d_k) + in;
  TO *dst = static_cast<TO *>(is_q ? a.d_q_out : is_v ? a.d_v_out : a.d_k_out) + out;

  float x[8];
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (live) Eight<TI>::load(src + d0, x);

  const uint32_t half = a.rot_dim / 2;
  const bool rotated = live && !is_v && d0 < a.rot_dim;
  const bool placed = a.rot_dim && !is_v;
  int32_t pos = placed ? a.d_positions[token] : 0;
  const bool lost = placed && (uint32_t)pos >= a.max_pos;
  if (lost) pos = 0;

  // pair index of value i: adjacent pairs (2p, 2p + 1), else (p, p + half)
  const bool adjacent = a.flags & ENC_ROPE_ADJACENT;
  float c[8], s[8];
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (rotated) {
    const float *row = a.d_table + (uint64_t)pos * a.rot_dim;
    for (int i = 0; i < 8; ++i) {
      const uint32_t d = d0 + i;
      if (d < a.rot_dim) {
        const uint32_t p = adjacent ? d / 2 : d < half ? d : d - half;
        c[i] = row[p];
        s[i] = row[half + p];
      }
    }
  }

  if (!(a.flags & ENC_QK_NO_NORM)) {
    float ss = 0.f;
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    for (uint32_t o = LANES / 2; o; o >>= 1) ss += __shfl_xor(ss, o);
    const float scale = 1.0f / sqrtf(ss / (float)a.head_dim + a.eps);
    if (!is_v)
      for (int i = 0; i < 8; ++i) x[i] *= scale;
  }
  const void *w = is_q ? a.d_q_weight : a.d_k_weight;
  if (live && !is_v && w) {
    float wv[8];
    load_weight(w, a.w_dtype, d0, wv);
    for (int i = 0; i < 8; ++i) x[i] *= wv[i];
  }

  if (adjacent) {
    for (int i = 0; i < 8; i += 2) {
      const float u = x[i], v = x[i + 1];
      x[i] = u * c[i] - v * s[i];
      x[i + 1] = v * c[i] + u * s[i];
    }
  } else if (a.rot_dim) {   // uniform over the launch
    float *mine = xs + threadIdx.x * 8;
    reinterpret_cast<f32x4 *>(mine)[0] = f32x4{x[0], x[1], x[2], x[3]};
    reinterpret_cast<f32x4 *>(mine)[1] = f32x4{x[4], x[5], x[6], x[7]};
    __syncthreads();
    if (rotated) {
      for (int i = 0; i < 8; ++i) {
        const uint32_t d = d0 + i;
        if (d < half)
          x[i] = x[i] * c[i] - mine[i + half] * s[i];
        else if (d < a.rot_dim)
          x[i] = x[i] * c[i] + mine[(int)i - (int)half] * s[i];
      }
    }
  }
  if (lost)
    for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
  if (live) Eight<TO>::store(dst + d0, x);
}

template <typename TI, typename TO>
void launch_lanes(const QkKernelArgs &k, hipStream_t s) {
  const uint32_t need = k.a.head_dim / 8;
  const uint32_t lanes = need <= 8 ? 8 : need <= 16 ? 16 : need <= 32 ? 32 : 64;
  const uint32_t per = kBlock / lanes;
  const dim3 grid((k.items + per - 1) / per), block(kBlock);
  switch (lanes) {
    case 8: hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, 8>), grid, block, 0, s, k); break;
    case 16: hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, 16>), grid, block, 0, s, k); break;
    case 32: hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, 32>), grid, block, 0, s, k); break;
    default: hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, 64>), grid, block, 0, s, k); break;
  }
}

template <typename TI>
void launch_out(const QkKernelArgs &k, hipStream_t s) {
  switch (k.a.out_dtype) {
    case 1: launch_lanes<TI, __bf16>(k, s); break;
    case 2: launch_lanes<TI, _Float16>(k, s); break;
    default: launch_lanes<TI, float>(k, s); break;
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkKernelArgs &k, hipStream_t s) {
  switch (k.a.in_dtype) {
    case 1: launch_out<__bf16>(k, s); break;
    case 2: launch_out<_Float16>(k, s); break;
    default: launch_out<float>(k, s); break;
  }
  return hipGetLastError();
}

}  // namespace enc
