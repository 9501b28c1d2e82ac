// verify_tree.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers (enc_verify_tree).
//
// The walk itself needs a target and a draft probability per child, gathered
// for all nodes at once. What it reads in bulk is one row of the target and
// of the draft for each node at which a child is rejected (the sum of
// max(r - q, 0)) or at which it ends (the draw). A lane keeps its part of the
// row in registers from the first rejection to the draw; without them, r is
// recomputed from p, q and the sums of the rejections before.
//
// Sums are whole numbers of 2^-40: exact, so neither the split over lanes,
// waves and workgroups nor its order shows in the answer.
//
// Bound: HBM traffic of those rows, and the rounds' latency. A row is split
// over up to 16 workgroups; every workgroup makes the same walk, sums its part of a row, publishes the
// sums of its waves' segments and takes those of the others. A workgroup that
// waits too long for the others (which may not have been scheduled) computes
// all segments by itself from then on, so no wait is unbounded. The
// workgroup whose segment holds the drawn token finds it. A sequence's
// workgroups are on one compute die, so that the words they exchange meet in
// its L2.
//
// Measured (fp32, 128256 values, us on the device): one sequence, a chain of 5:
// 12.9; 32 trees of 16 nodes: 45, with 33 MB of rows read (7 at a copy's rate):
// the rounds, one per rejection, each with an exchange, are most of it.
#include "step_common.h"

#include <cstdlib>

namespace enc {
namespace {

constexpr uint32_t kThreadsV = 1024, kWaves = kThreadsV / 64;
constexpr uint32_t kMaxGroups = 16, kMaxSegments = kMaxGroups * kWaves;
constexpr uint32_t kMaxNodes = ENC_TREE_MAX_NODES;
typedef unsigned long long u64;

__device__ __forceinline__ float clamp01(float x) { return __builtin_amdgcn_fmed3f(x, 0.f, 1.f); }   // NaN: 0

// x (up to 1) in whole multiples of 2^-40, ties to even. In steps of 2^-20,
// whose remainder is exact, and which leave nothing to round above 2^-16.
__device__ __forceinline__ u64 mass(float x) {
  const float y = x * 1099511627776.f;
  const float h = truncf(y * (1.f / 1048576.f));
  return ((u64)(uint32_t)h << 20) + (uint32_t)rintf(fmaf(-h, 1048576.f, y));
}

// Four of them; as almost always, none reaches 2^-8, and each fits 32 bits.
__device__ __forceinline__ u64 mass4(float a, float b, float c, float d) {
  if (__any(fmaxf(fmaxf(a, b), fmaxf(c, d)) >= 0.00390625f)) return (mass(a) + mass(b)) + (mass(c) + mass(d));
  auto small = [](float x) { return (u64)(uint32_t)rintf(x * 1099511627776.f); };
  return (small(a) + small(b)) + (small(c) + small(d));
}

template <typename T> __device__ __forceinline__ float value_at(const void *row, uint32_t i);
template <> __device__ __forceinline__ float value_at<float>(const void *row, uint32_t i) {
  return clamp01(static_cast<const float *>(row)[i]);
}
template <> __device__ __forceinline__ float value_at<__bf16>(const void *row, uint32_t i) {
  return clamp01(__uint_as_float((uint32_t)static_cast<const uint16_t *>(row)[i] << 16));
}
template <> __device__ __forceinline__ float value_at<_Float16>(const void *row, uint32_t i) {
  return clamp01((float)static_cast<const _Float16 *>(row)[i]);
}

__device__ __forceinline__ u64 wave_sum(u64 v) {
  for (uint32_t o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The rejections at the current node.
struct Rejections {
  uint32_t n;                 // how many
  float sum[kMaxNodes];       // fp32 sum of max(r - q, 0) after each; 0: r was left as it was
  int32_t token[kMaxNodes];
};

// r_i after the first n rejections, and in `left` what it is a multiple of:
// the last nonempty difference (p_i if there is none).
template <bool POINT>
__device__ __forceinline__ float residual(float p, float q, int32_t i, const Rejections &x, uint32_t n,
                                          float &left) {
  float r = p;
  left = p;
  for (uint32_t k = 0; k < n; ++k) {
    const float s = x.sum[k];
    if (s > 0.f) {
      const float qk = POINT ? (x.token[k] == i ? 1.f : 0.f) : q;
      left = fmaxf(r - qk, 0.f);
      r = left / s;
    }
  }
  return r;
}

// Four consecutive values, in one load.
template <typename T>
__device__ __forceinline__ void four_at(const void *row, uint32_t i, float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + i);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + i);
    x[0] = half_of<T>(v.x, 0), x[1] = half_of<T>(v.x, 1), x[2] = half_of<T>(v.y, 0), x[3] = half_of<T>(v.y, 1);
  }
  for (int e = 0; e < 4; ++e) x[e] = clamp01(x[e]);
}

// EPT: values of a row a lane keeps in registers, so that the rejections at a
// node and the draw from it read the row once; 0: rows are read each time.
template <typename T, bool POINT, uint32_t EPT>
__global__ __launch_bounds__(kThreadsV) void k_verify(VerifyKernelArgs k) {
  const enc_verify_args &a = k.a;
  __shared__ int32_t token[kMaxNodes];
  __shared__ float u[kMaxNodes], pc[kMaxNodes], qc[kMaxNodes];
  __shared__ int32_t path[kMaxNodes];
  __shared__ Rejections rej;
  __shared__ u64 totals[kMaxSegments], kept[kMaxSegments];
  __shared__ u64 scan[kWaves];
  __shared__ uint32_t alone;

  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // a sequence's workgroups differ by 8, which places them on one compute die
  // (workgroups go to the 8 dies in turn): their words meet in its L2
  const uint32_t G = k.groups, id8 = blockIdx.x >> 3, set = id8 / G;
  const uint32_t b = set * 8 + (blockIdx.x & 7), g = id8 - set * G;
  if (b >= a.batch) return;
  const uint32_t segments = G * kWaves;
  const uint32_t T_ = a.nodes, V = a.vocab;
  int32_t live = a.d_nodes ? a.d_nodes[b] : (int32_t)T_;
  live = max(0, min(live, (int32_t)T_));
  const char *target = static_cast<const char *>(a.d_target) + (uint64_t)b * a.target_batch * sizeof(T);
  const char *draft = static_cast<const char *>(a.d_draft) + (POINT ? 0 : (uint64_t)b * a.draft_batch * sizeof(T));
  const uint64_t trow = a.target_node * sizeof(T), drow = a.draft_node * sizeof(T);

  // every node's parent, in registers of every wave: node 64 j + lane
  int32_t parent[kMaxNodes / 64];
#pragma unroll
  for (uint32_t j = 0; j < kMaxNodes / 64; ++j) {
    const int32_t i = (int32_t)(64 * j + lane);
    parent[j] = i >= 1 && i < live ? a.d_parents[(uint64_t)b * T_ + i] : -1;
    if (parent[j] >= i) parent[j] = -1;
  }
  if (tid < T_) {
    const int32_t i = (int32_t)tid;
    u[tid] = a.d_u[(uint64_t)b * T_ + tid];
    path[tid] = -1;
    float p = 0.f, q = 0.f;
    int32_t x = -1;
    if (i >= 1 && i < live) {
      const int32_t up = a.d_parents[(uint64_t)b * T_ + i];
      x = a.d_tokens[(uint64_t)b * T_ + i];
      if ((uint32_t)x >= V) x = -1;
      if (up >= 0 && up < i && x >= 0) {
        p = value_at<T>(target + up * trow, (uint32_t)x);
        q = POINT ? 1.f : value_at<T>(draft + up * drow, (uint32_t)x);
      }
    }
    token[tid] = x;
    pc[tid] = p;
    qc[tid] = q;
  }
  if (tid == 0) {
    rej.n = 0;
    alone = 0;
  }
  __syncthreads();

  u64 total = 0;             // of what `kept` holds the segments of
  uint32_t round = 0;
  bool solo = false;         // this workgroup no longer waits for the others

  // this lane's values of the current node's row: chunk c of 4 holds elements
  // seg0 + 256 c + 4 lane .. + 3
  constexpr uint32_t N = EPT ? EPT : 4;
  float r[N], q[N], left[N];
  const uint32_t seg0 = (g * kWaves + wave) * k.segment;
  int32_t held = -1;         // the node whose row they are
  // After a rejection `left` is the difference, and `over` its sum: r becomes
  // left / over only if another child is rejected here.
  float over = 0.f;
  auto hold = [&](uint32_t cur, bool with_q) {
    if (held == (int32_t)cur) return;
    held = (int32_t)cur;
    over = 0.f;
    const char *prow = target + cur * trow, *qrow = draft + cur * drow;
    // 4 values in a load where the wave's part of both rows allows it
    const bool whole = ((reinterpret_cast<uintptr_t>(prow) | (POINT ? 0 : reinterpret_cast<uintptr_t>(qrow))) &
                        (4 * sizeof(T) - 1)) == 0 && seg0 + 64 * N <= V;
    if (whole) {
#pragma unroll
      for (uint32_t c = 0; c < N; c += 4) {
        const uint32_t i = seg0 + 64 * c + 4 * lane;
        float p4[4], q4[4] = {0.f, 0.f, 0.f, 0.f};
        four_at<T>(prow, i, p4);
        if (!POINT && with_q) four_at<T>(qrow, i, q4);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) r[c + e] = p4[e], q[c + e] = q4[e];
      }
    } else {
#pragma unroll
      for (uint32_t j = 0; j < N; ++j) {
        const uint32_t i = seg0 + 64 * (j & ~3u) + 4 * lane + (j & 3u);
        r[j] = i < V ? value_at<T>(prow, i) : 0.f;
        q[j] = !POINT && with_q && i < V ? value_at<T>(qrow, i) : 0.f;
      }
    }
#pragma unroll
    for (uint32_t j = 0; j < N; ++j) left[j] = r[j];
  };
  auto index_of = [&](uint32_t j) { return seg0 + 64 * (j & ~3u) + 4 * lane + (j & 3u); };
  auto settle = [&] {
    if (!(over > 0.f)) return;
#pragma unroll
    for (uint32_t j = 0; j < N; ++j) {
      r[j] = left[j] / over;
      if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // a few quotients at a time: registers
    }
    over = 0.f;
  };
  auto reject = [&](float sum, int32_t x) {
#pragma unroll
    for (uint32_t j = 0; j < N; ++j)
      left[j] = fmaxf(r[j] - (POINT ? ((int32_t)index_of(j) == x ? 1.f : 0.f) : q[j]), 0.f);
    over = sum;
  };

  // Sums of `left` over every segment of the current node's row, after n
  // rejections, into totals[]; returns their sum. With `pending`, the n-th
  // rejection's own sum is what is being computed: r - q is taken of r.
  auto sum_row = [&](uint32_t cur, uint32_t n, bool pending) -> u64 {
    const char *prow = target + cur * trow, *qrow = draft + cur * drow;
    const int32_t ptoken = pending ? rej.token[n] : -1;
    auto segment_sum = [&](uint32_t seg) -> u64 {
      const uint64_t lo = (uint64_t)seg * k.segment;
      u64 acc = 0;
      if (lo < V) {
        const uint32_t hi = (uint32_t)(lo + k.segment < V ? lo + k.segment : V);
        for (uint32_t i0 = (uint32_t)lo; i0 < hi; i0 += 256) {
          float p[4], q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t i = i0 + 64 * e + lane;
            p[e] = i < hi ? value_at<T>(prow, i) : 0.f;
            q[e] = !POINT && i < hi ? value_at<T>(qrow, i) : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t i = (int32_t)(i0 + 64 * e + lane);
            float left;
            const float r = residual<POINT>(p[e], q[e], i, rej, n, left);
            if (pending) left = fmaxf(r - (POINT ? (i == ptoken ? 1.f : 0.f) : q[e]), 0.f);
            acc += mass(left);
          }
        }
      }
      return wave_sum(acc);
    };
    auto own_sum = [&]() -> u64 {
      if (!EPT) return segment_sum(g * kWaves + wave);
      hold(cur, pending);
      if (pending) settle();
      u64 acc = 0;
#pragma unroll
      for (uint32_t j = 0; j < N; j += 4) {
        float d[4];
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const float qk = POINT ? ((int32_t)index_of(j + e) == ptoken ? 1.f : 0.f) : q[j + e];
          d[e] = pending ? fmaxf(r[j + e] - qk, 0.f) : left[j + e];
        }
        acc += mass4(d[0], d[1], d[2], d[3]);
        __builtin_amdgcn_sched_barrier(0);
      }
      return wave_sum(acc);
    };
    if (G > 1 && !solo) {
      // a sum and the round it belongs to (modulo 3, plus 1) in one word, so a
      // word is there or not; two slots in turn: nobody writes round r + 2
      // before everybody has published r + 1, and so has read r
      u64 *out = k.totals + ((uint64_t)b * 2 + (round & 1)) * segments;
      const u64 tag = (u64)(round % 3 + 1) << 62;
      const u64 t = own_sum();
      if (lane == 0)
        __hip_atomic_store(&out[g * kWaves + wave], t | tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (wave * 64 < segments) {
        u64 got = tag;
        uint32_t polls = 0;
        while (true) {
          if (tid < segments) got = __hip_atomic_load(&out[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          if (__all(got >> 62 == tag >> 62)) break;
          if (polls++ >= k.spins) {
            if (lane == 0) alone = 1;
            break;
          }
          __builtin_amdgcn_s_sleep(1);
        }
        if (tid < segments) totals[tid] = got & ~(3ull << 62);
      }
      __syncthreads();
      solo = alone;
    }
    if (G == 1) {
      const u64 t = own_sum();
      if (lane == 0) totals[wave] = t;
    } else if (solo) {
      for (uint32_t s = wave; s < segments; s += kWaves) {
        const u64 t = segment_sum(s);
        if (lane == 0) totals[s] = t;
      }
    }
    ++round;
    __syncthreads();
    const u64 mine = tid < segments ? totals[tid] : 0;
    const u64 ws = wave_sum(mine);
    if (lane == 0) scan[wave] = ws;
    __syncthreads();
    u64 all = 0;
    for (uint32_t w = 0; w < kWaves; ++w) all += scan[w];
    __syncthreads();
    return all;
  };

  // ---- the walk: the same in every thread
  uint32_t cur = 0, count = 0;
  bool have = false;          // kept[] and total hold the current node's `left`
  if (live > 0) {
    if (tid == 0) path[0] = 0;
    count = 1;
    int32_t last = 0;         // children up to here are done with
    while (true) {
      uint32_t c = 0;
#pragma unroll
      for (uint32_t j = 0; j < kMaxNodes / 64; ++j) {
        const int32_t i = (int32_t)(64 * j + lane);
        const uint64_t m = __ballot(parent[j] == (int32_t)cur && i > last);
        if (!c && m) c = 64 * j + (uint32_t)__builtin_ctzll(m);
      }
      if (!c && have) break;
      const int32_t x = c ? token[c] : -1;
      const uint32_t n = rej.n;
      if (c) {
        last = (int32_t)c;
        if (x < 0) continue;
        float l;
        if (u[c] * qc[c] < residual<POINT>(pc[c], qc[c], x, rej, n, l)) {
          cur = c;
          have = false;
          __syncthreads();
          if (tid == 0) {
            path[count] = (int32_t)c;
            rej.n = 0;
          }
          ++count;
          __syncthreads();
          continue;
        }
        __syncthreads();
        if (tid == 0) rej.token[n] = x;
        __syncthreads();
      }
      // c was rejected, or there is no child left and no sum yet
      const u64 sum = sum_row(cur, n, c != 0);
      if (sum || !c) {
        if (tid < segments) kept[tid] = totals[tid];
        total = sum;
        have = true;
      }
      if (!c) {
        __syncthreads();
        break;
      }
      const float sum32 = (float)sum * (1.f / 1099511627776.f);
      if (EPT && !solo && sum) reject(sum32, x);
      if (tid == 0) {
        rej.sum[n] = sum32;
        rej.n = n + 1;
      }
      __syncthreads();
    }
  }

  if (g == 0) {
    for (uint32_t i = tid; i < T_; i += kThreadsV) a.d_path[(uint64_t)b * T_ + i] = path[i];
    if (tid == 0) {
      a.d_count[b] = (int32_t)count;
      if (total == 0) a.d_token[b] = -1;
    }
  }
  if (total) {
    // the segment in which the running sum passes the goal, then the element
    const float u0 = u[0];
    const uint32_t point = u0 > 0.f ? (uint32_t)(fminf(u0, 1.f - 1.f / 16777216.f) * 16777216.f) : 0u;
    const u64 goal = (total >> 24) * point + (((total & 0xFFFFFFull) * point) >> 24);
    auto block_excl = [&](u64 v) -> u64 {
      u64 incl = v;
      for (uint32_t o = 1; o < 64; o <<= 1) {
        const u64 t = __shfl_up(incl, o);
        if (lane >= o) incl += t;
      }
      __syncthreads();
      if (lane == 63) scan[wave] = incl;
      __syncthreads();
      u64 before = 0;
      for (uint32_t w = 0; w < wave; ++w) before += scan[w];
      return before + incl - v;
    };
    const u64 mine = tid < segments ? kept[tid] : 0;
    const u64 before = block_excl(mine);
    __shared__ uint32_t hit;
    __shared__ u64 hit_before;
    if (before <= goal && goal < before + mine) {
      hit = tid;
      hit_before = before;
    }
    __syncthreads();
    const uint32_t seg = hit;
    if (EPT && !solo) {
      if (seg == g * kWaves + wave) {
        u64 at = hit_before;
#pragma unroll
        for (uint32_t c = 0; c < N; c += 4) {
          u64 w[4], four = 0;
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) four += w[e] = mass(left[c + e]);
          u64 incl = four;
          for (uint32_t o = 1; o < 64; o <<= 1) {
            const u64 t = __shfl_up(incl, o);
            if (lane >= o) incl += t;
          }
          u64 from = at + incl - four;
          if (from <= goal && goal < from + four) {
            uint32_t e = 0;
            while (from + w[e] <= goal) from += w[e++];
            a.d_token[b] = (int32_t)(index_of(c) + e);
          }
          at += __shfl(incl, 63);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else if (seg / kWaves == g) {
      const char *prow = target + cur * trow, *qrow = draft + cur * drow;
      const uint32_t lo = seg * k.segment, hi = min(lo + k.segment, V);
      const uint32_t per = (k.segment + kThreadsV - 1) / kThreadsV;
      auto left_at = [&](uint32_t i) -> u64 {
        float l;
        residual<POINT>(value_at<T>(prow, i), POINT ? 0.f : value_at<T>(qrow, i), (int32_t)i, rej, rej.n, l);
        return mass(l);
      };
      const uint32_t i0 = lo + tid * per;
      u64 sum = 0;
      for (uint32_t i = i0; i < min(i0 + per, hi); ++i) sum += left_at(i);
      u64 at = hit_before + block_excl(sum);
      if (at <= goal && goal < at + sum) {
        for (uint32_t i = i0; i < hi; ++i) {
          at += left_at(i);
          if (at > goal) {
            a.d_token[b] = (int32_t)i;
            break;
          }
        }
      }
    }
  }

  // the last workgroup of a sequence leaves its words at zero for the next call
  if (G > 1) {
    __shared__ uint32_t order;
    // A workgroup that waited to the end has read its own words back. One that
    // gave up has not: they must have arrived before it counts as through, or
    // the last one's zeros could be overtaken.
    if (solo) __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    __syncthreads();
    if (tid == 0) order = __hip_atomic_fetch_add(&k.done[b], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (order == G - 1) {
      for (uint32_t i = tid; i < 2 * segments; i += kThreadsV)
        __hip_atomic_store(&k.totals[(uint64_t)b * 2 * segments + i], 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (tid == 0) __hip_atomic_store(&k.done[b], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

template <typename T, bool POINT>
void launch_kept(const VerifyKernelArgs &k, hipStream_t s) {
  const dim3 grid((k.a.batch + 7) / 8 * 8 * k.groups), block(kThreadsV);
  switch (k.segment) {
    case 64 * 4: hipLaunchKernelGGL((k_verify<T, POINT, 4>), grid, block, 0, s, k); break;
    case 64 * 8: hipLaunchKernelGGL((k_verify<T, POINT, 8>), grid, block, 0, s, k); break;
    case 64 * 16: hipLaunchKernelGGL((k_verify<T, POINT, 16>), grid, block, 0, s, k); break;
    default: hipLaunchKernelGGL((k_verify<T, POINT, 0>), grid, block, 0, s, k); break;
  }
}

template <typename T>
void launch_t(const VerifyKernelArgs &k, hipStream_t s) {
  if (k.a.d_draft)
    launch_kept<T, false>(k, s);
  else
    launch_kept<T, true>(k, s);
}

}  // namespace

// A lane keeps 4, 8 or 16 values of a row, a workgroup 4096, 8192 or 16384; of
// these the smallest with which the workgroups of all sequences find a
// compute unit each, and a sequence has at most 16 (whose waves' sums then fit
// a thread each). us with 4, 8, 16 values: one sequence, 32000 words 12.8, 13.8,
// 16.7; one, 128256 words (4: too many workgroups) -, 13.7, 16.7; 16 -, 23.4,
// 26.1; 32 trees, which with 8 would be 512 workgroups, -, 58, 44. Rows above 16 x 16384 values are read again each time.
VerifyPlan plan_verify_tree(uint32_t batch, uint32_t vocab) {
  VerifyPlan p;
  uint32_t ept = 4;
  while (ept < 16) {
    const uint32_t g = (vocab + kWaves * 64 * ept - 1) / (kWaves * 64 * ept);
    if (g <= kMaxGroups && (uint64_t)g * batch <= 256) break;
    ept *= 2;
  }
  p.segment = 64 * ept;
  p.groups = (vocab + kWaves * p.segment - 1) / (kWaves * p.segment);
  if (p.groups > kMaxGroups) {
    p.groups = kMaxGroups;
    p.segment = ((vocab + kMaxSegments - 1) / kMaxSegments + 255) & ~255u;
  }
  const uint32_t segments = p.groups * kWaves;
  p.totals_bytes = align_up(8ull * batch * 2 * segments, 256);
  p.done_bytes = align_up(4ull * batch, 256);
  return p;
}

hipError_t launch_verify_tree(const VerifyKernelArgs &k, hipStream_t s) {
  switch (k.a.dtype) {
    case 1: launch_t<__bf16>(k, s); break;
    case 2: launch_t<_Float16>(k, s); break;
    default: launch_t<float>(k, s); break;
  }
  return hipGetLastError();
}

}  // namespace enc
