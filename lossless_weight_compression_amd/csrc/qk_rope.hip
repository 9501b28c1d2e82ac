// qk_rope.hip -- norms of query and key heads, rotary embedding and type
// conversion in one pass (enc_qk_norm_rope).
//
// y = x rsqrt(mean(x^2) + eps) w over a head, then the first rot_dim values
// turned pairwise by the token's angles. Every value is read once, held in
// fp32 and rounded once. The bound is HBM traffic (about 8 flops per value):
// a head of D values is held by D/8 lanes (rounded up to a power of two, so
// its sum is a butterfly inside one wave), 8 consecutive values each, which
// makes every load and store 16 bytes or more per lane. Values are exchanged
// between the two halves of a head through LDS, within the wave.
//
// Measured (us on the device): 8192 tokens of 48 heads of 128, fp32 in, BF16
// out (306 MB): 60, 5.1 TB/s, where a large copy reaches 4.9; 792 tokens of 24
// heads of 64 in BF16: 4.6; one token: 3.1 of a call's 12 (the rest is the
// host's).
#include "step_common.h"

#include <algorithm>

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

// R heads of one token to a lane (the same values of each), so the token's
// angles are read once for them and R rows are on their way at a time. VEC:
// the angles of a lane's values lie in runs of 4, aligned.
template <typename TI, typename TO, uint32_t LANES, uint32_t R, bool VEC>
__global__ __launch_bounds__(kBlock) void k_qk_norm_rope(QkKernelArgs k) {
  const enc_qk_args &a = k.a;
  constexpr uint32_t kHeads = kBlock / LANES;   // heads of a workgroup, R times
  __shared__ __align__(16) float xs[kBlock * 8];
  const uint32_t chunk = threadIdx.x % LANES, d0 = chunk * 8;
  const uint32_t turn = k.blocks.quot(blockIdx.x), block = blockIdx.x - turn * k.blocks.d;
  const uint32_t token = k.token0 + turn;
  const uint32_t first = block * (kHeads * R) + threadIdx.x / LANES;
  const uint32_t rotated_heads = a.q_heads + a.kv_heads;
  const bool in_head = d0 < a.head_dim;

  float x[R][8];
#pragma unroll
  for (uint32_t i = 0; i < R; ++i) {
    const uint32_t head = first + i * kHeads;
    const bool is_q = head < a.q_heads, is_v = head >= rotated_heads;
    const uint32_t h = is_q ? head : is_v ? head - rotated_heads : head - a.q_heads;
    const uint64_t at = is_q   ? token * a.q_token + h * a.q_head
                        : is_v ? token * a.v_token + h * a.v_head
                               : token * a.k_token + h * a.k_head;
    const TI *src = static_cast<const TI *>(is_q ? a.d_q : is_v ? a.d_v : a.d_k) + at;
    for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    if (head < k.heads && in_head) Eight<TI>::load(src + d0, x[i]);
  }

  const uint32_t half = a.rot_dim / 2;
  const bool turns = in_head && d0 < a.rot_dim;
  const bool adjacent = a.flags & ENC_ROPE_ADJACENT;
  int32_t pos = a.rot_dim ? a.d_positions[token] : 0;
  const bool lost = a.rot_dim && (uint32_t)pos >= a.max_pos;
  if (lost) pos = 0;
  // value e's angle: pair (d0 + e) / 2 if adjacent (4 of them), else d0 + e, less
  // half in the second half
  float c[8], s[8];
  for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  if (turns) {
    const float *row = a.d_table + (uint64_t)pos * a.rot_dim;
    if constexpr (VEC) {
      const uint32_t p = adjacent ? d0 / 2 : d0 < half ? d0 : d0 - half;
      const f32x4 c0 = *reinterpret_cast<const f32x4 *>(row + p), s0 = *reinterpret_cast<const f32x4 *>(row + half + p);
      f32x4 c1 = c0, s1 = s0;
      if (!adjacent) {
        c1 = *reinterpret_cast<const f32x4 *>(row + p + 4);
        s1 = *reinterpret_cast<const f32x4 *>(row + half + p + 4);
      }
      for (int e = 0; e < 4; ++e) {
        if (adjacent) {
          c[2 * e] = c[2 * e + 1] = c0[e];
          s[2 * e] = s[2 * e + 1] = s0[e];
        } else {
          c[e] = c0[e], c[4 + e] = c1[e];
          s[e] = s0[e], s[4 + e] = s1[e];
        }
      }
    } else {
      for (int e = 0; e < 8; ++e) {
        const uint32_t d = d0 + e;
        if (d < a.rot_dim) {
          const uint32_t p = adjacent ? d / 2 : d < half ? d : d - half;
          c[e] = row[p];
          s[e] = row[half + p];
        }
      }
    }
  }

#pragma unroll
  for (uint32_t i = 0; i < R; ++i) {
    const uint32_t head = first + i * kHeads;
    const bool live = head < k.heads && in_head;
    const bool is_q = head < a.q_heads, is_v = head >= rotated_heads;
    if (!(a.flags & ENC_QK_NO_NORM)) {
      float ss = 0.f;
      for (int e = 0; e < 8; ++e) ss = fmaf(x[i][e], x[i][e], ss);
#pragma unroll
      for (uint32_t o = LANES / 2; o; o >>= 1) ss += __shfl_xor(ss, o);
      const float scale = 1.0f / sqrtf(ss / (float)a.head_dim + a.eps);
      if (!is_v)
        for (int e = 0; e < 8; ++e) x[i][e] *= scale;
    }
    const void *w = is_q ? a.d_q_weight : a.d_k_weight;
    if (live && !is_v && w) {
      float wv[8];
      load_weight(w, a.w_dtype, d0, wv);
      for (int e = 0; e < 8; ++e) x[i][e] *= wv[e];
    }
    if (adjacent) {
      if (turns && !is_v) {
        for (int e = 0; e < 8; e += 2) {
          if (!VEC && d0 + e >= a.rot_dim) continue;   // 0 times an infinity is no number
          const float u = x[i][e], v = x[i][e + 1];
          x[i][e] = u * c[e] - v * s[e];
          x[i][e + 1] = v * c[e] + u * s[e];
        }
      }
    } else if (a.rot_dim) {   // uniform over the launch
      // the other half's values through LDS; a head's lanes are one wave's, whose
      // LDS operations keep their order
      float *mine = xs + threadIdx.x * 8;
      reinterpret_cast<f32x4 *>(mine)[0] = f32x4{x[i][0], x[i][1], x[i][2], x[i][3]};
      reinterpret_cast<f32x4 *>(mine)[1] = f32x4{x[i][4], x[i][5], x[i][6], x[i][7]};
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (turns && !is_v) {
        if constexpr (VEC) {
          const float *other = d0 < half ? mine + half : mine - half;
          const f32x4 o0 = reinterpret_cast<const f32x4 *>(other)[0], o1 = reinterpret_cast<const f32x4 *>(other)[1];
          for (int e = 0; e < 8; ++e) {
            const float turn = s[e] * (e < 4 ? o0[e & 3] : o1[e & 3]);
            x[i][e] = d0 < half ? x[i][e] * c[e] - turn : x[i][e] * c[e] + turn;
          }
        } else {
          for (int e = 0; e < 8; ++e) {
            const uint32_t d = d0 + e;
            if (d < half)
              x[i][e] = x[i][e] * c[e] - mine[e + half] * s[e];
            else if (d < a.rot_dim)
              x[i][e] = x[i][e] * c[e] + mine[e - (int)half] * s[e];
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (lost && !is_v)
      for (int e = 0; e < 8; ++e) x[i][e] = __builtin_nanf("");
    if (live) {
      const uint32_t h = is_q ? head : is_v ? head - rotated_heads : head - a.q_heads;
      const uint64_t at = is_q   ? token * a.q_out_token + h * a.q_out_head
                          : is_v ? token * a.v_out_token + h * a.v_out_head
                                 : token * a.k_out_token + h * a.k_out_head;
      TO *dst = static_cast<TO *>(is_q ? a.d_q_out : is_v ? a.d_v_out : a.d_k_out) + at;
      Eight<TO>::store(dst + d0, x[i]);
    }
  }
}

// Three heads to a lane once that still gives every compute unit eight
// workgroups, one below, where latency counts (us a call of ten in a graph, three
// and one: 8192 tokens of 48 heads of 128 65.4, 67.6; 1024: 10.4, 10.3; 792 of 24
// heads of 64 5.6, 4.9; 256 of 48 heads of 128 6.3, 4.6).
template <typename TI, typename TO, uint32_t LANES>
void launch_heads(QkKernelArgs k, hipStream_t s) {
  constexpr uint32_t per = kBlock / LANES;
  const uint32_t thirds = (k.heads + 3 * per - 1) / (3 * per);
  const bool many = k.vec && (uint64_t)thirds * k.a.tokens >= 2048;
  const uint32_t blocks = many ? thirds : (k.heads + per - 1) / per;
  k.blocks = FastDiv::of(blocks);
  // a grid holds fewer than 2^32 threads
  const uint32_t most = (1u << 23) / blocks;
  for (k.token0 = 0; k.token0 < k.a.tokens; k.token0 += most) {
    const dim3 grid(blocks * std::min(most, k.a.tokens - k.token0)), block(kBlock);
    if (many)
      hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, LANES, 3, true>), grid, block, 0, s, k);
    else if (k.vec)
      hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, LANES, 1, true>), grid, block, 0, s, k);
    else
      hipLaunchKernelGGL((k_qk_norm_rope<TI, TO, LANES, 1, false>), grid, block, 0, s, k);
  }
}

template <typename TI, typename TO>
void launch_lanes(const QkKernelArgs &k, hipStream_t s) {
  const uint32_t need = k.a.head_dim / 8;
  if (need <= 8)
    launch_heads<TI, TO, 8>(k, s);
  else if (need <= 16)
    launch_heads<TI, TO, 16>(k, s);
  else if (need <= 32)
    launch_heads<TI, TO, 32>(k, s);
  else
    launch_heads<TI, TO, 64>(k, s);
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
