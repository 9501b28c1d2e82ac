// tree_attention.hip -- attention of a tree's nodes over a paged cache and
// the tree itself (enc_tree_attention).
//
// One pass over the keys with a running maximum m and sum l per query row:
// o = sum_j e^(s_j - m) v_j / l, s_j = scale q.k_j. The query rows
// that share a KV head (nodes x heads of its group) are one matrix, so every
// key and value is read once for all of them: HBM traffic of the cache is the
// bound, until some 200 rows share a KV head.
//
// Nothing of K or V passes through LDS. A wave takes strips of 32 keys and
// computes S^T = K Q^T and O^T += V^T P^T with v_mfma 16x16x32:
//  * K: lane l holds 8 consecutive values of key l % 16, so fragments are
//    loaded from the rows as they lie, 16 bytes a lane.
//  * S^T leaves lane l with keys 4 (l / 16) + i of query row l % 16. The sum
//    over keys in P V may run in any order, so key 16 t + 4 g + i is made
//    contraction index 8 g + 4 t + i: then these registers, rounded, are the
//    P^T fragment, with no exchange between lanes.
//  * V: lane l loads, of its group's 8 keys, values (l % 16) C .. + C - 1
//    (C = 8 for 128 values: whole rows per 16 lanes) and transposes them in
//    registers, one byte permute per output dword. Row m of V^T fragment f
//    then stands for value m C + f, and lane l's accumulators hold runs of
//    C consecutive values of its row, stored 16 bytes at a time.
//  * m and l belong to the lane's own query row; rescaling needs no exchange.
// P is rounded to the values' type (its relative error, 2^-9 for BF16, is
// that of the result's own rounding); sums, m, l and o are fp32. A row's m
// only moves when a strip exceeds it by more than 8 (a factor of 2^8, far
// inside fp32 and both 16-bit ranges), which makes rescaling rare.
//
// The keys of a (sequence, KV head) are split over workgroups so that a few
// long sequences fill the device too; the parts are joined by a second
// kernel, in order. The four waves of a workgroup hold different rows (64
// each) or different strips, joined through LDS at the end.
#include "step_common.h"

namespace enc {
namespace {

constexpr float kLowest = -3.402823466e38f;   // finite: differences with it are not NaN
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.0f * kLn2;

// e^x. Scores stay in natural units until here: the difference of two finite
// scores does not overflow, a score times log2(e) may.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
constexpr uint32_t kWavesA = 4;

template <typename T> struct Half;
template <> struct Half<__bf16> {
  static constexpr uint32_t kExp = 0x7F80u;
  static constexpr float kLift = 0.f;
  static __device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};
template <> struct Half<_Float16> {
  static constexpr uint32_t kExp = 0x7C00u;
  // P is held 2^6 larger (at most 2^14): FP16 loses precision below 2^-14, and
  // many keys of little weight together still count
  static constexpr float kLift = 6.f * kLn2;
  static __device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
};

// Strips a workgroup takes: an equal share, whole rounds of its key ways.
__device__ __forceinline__ uint32_t split_chunk(uint32_t strips, uint32_t splits, uint32_t ways) {
  const uint32_t c = (strips + splits - 1) / splits;
  return max((c + ways - 1) / ways * ways, ways);
}

struct Seq {
  uint32_t len, live, strips_ctx, strips;
  const int32_t *table;
};

__device__ __forceinline__ Seq sequence_of(const enc_tree_attention_args &a, uint32_t b) {
  Seq q;
  const uint32_t s = a.d_seqs ? (uint32_t)a.d_seqs[b] : b;
  const uint64_t room = (uint64_t)a.max_pages * a.page_size;
  int32_t len = s < a.max_seqs ? a.d_lens[s] : 0;
  len = max(len, 0);
  q.len = (uint64_t)len > room ? (uint32_t)room : (uint32_t)len;
  q.table = a.d_table + (uint64_t)(s < a.max_seqs ? s : 0) * a.max_pages;
  int32_t live = a.d_nodes ? a.d_nodes[b] : (int32_t)a.nodes;
  q.live = (uint32_t)max(0, min(live, (int32_t)a.nodes));
  q.strips_ctx = (q.len + 31) / 32;
  q.strips = q.strips_ctx + (q.live + 31) / 32;
  return q;
}

// DP: head_dim rounded up to what the fragments hold; EXACT: equal to it.
// U: 16-row units of a wave.
template <typename T, int DP, int U, bool EXACT>
__global__ __launch_bounds__(256) void k_tree_attention(TreeAttnArgs k, uint32_t row_ways) {
  constexpr int KS = DP / 32;                   // k steps of Q K^T
  constexpr int C = DP >= 128 ? 8 : DP / 16;    // consecutive values a lane transposes
  constexpr int NH = DP / (16 * C);             // groups of 16 C values
  constexpr int NREG = U * NH * C * 4;          // accumulators a lane holds
  const enc_tree_attention_args &a = k.a;
  __shared__ float joint[2 * (NREG + 2 * U) * 64];

  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t l16 = lane & 15, g4 = lane >> 4;
  const uint32_t D = a.head_dim;

  // workgroups of one (sequence, split, head) differ in 8, so they meet in one
  // compute die's L2 (workgroups go to the 8 dies in turn)
  const uint32_t groups = a.batch * k.splits * a.kv_heads;
  const uint32_t id8 = blockIdx.x >> 3;
  const uint32_t grp = id8 / k.row_tiles * 8 + (blockIdx.x & 7), rt = id8 % k.row_tiles;
  if (grp >= groups) return;
  const uint32_t h = grp % a.kv_heads, bs = grp / a.kv_heads, split = bs % k.splits, b = bs / k.splits;
  const Seq q = sequence_of(a, b);
  const uint32_t ways = kWavesA / row_ways, rw = wave % row_ways, kw = wave / row_ways;
  const uint32_t chunk = split_chunk(q.strips, k.splits, ways);
  const uint32_t lo = split * chunk, hi = min(lo + chunk, q.strips);
  if (lo >= q.strips && k.splits > 1) return;   // nothing for this split; the join does not look for it

  // ---- Q fragments: query row l % 16 of each unit, 8 values per k step
  const uint32_t row0 = (rt * row_ways + rw) * (U * 16) + l16;
  uint4 qf[U][KS];
  uint32_t node[U];
  bool alive[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = row0 + 16 * u;
    const uint32_t rr = min(r, k.rows - 1);
    node[u] = k.group.quot(rr);
    const uint32_t head = h * k.group.d + (rr - node[u] * k.group.d);
    alive[u] = r < k.rows && node[u] < q.live;
    const T *p = static_cast<const T *>(a.d_q) + b * a.q_batch + node[u] * a.q_node + head * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t d = 32 * s + 8 * g4;
      qf[u][s] = make_uint4(0, 0, 0, 0);
      if (alive[u] && (EXACT || d < D)) qf[u][s] = *reinterpret_cast<const uint4 *>(p + d);
    }
  }

  f32x4 o[U][NH][C];
  float m[U], l[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = kLowest;
    l[u] = 0.f;
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int f = 0; f < C; ++f) o[u][x][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // ---- strips: cached keys, then the tree's own; one strip's registers, each
  // half loaded again as soon as it has been used
  uint4 kf[2][KS];
  uint32_t vr[8][NH][C / 2];
  const uint4 *kc = static_cast<const uint4 *>(a.d_k_cache) + h * (a.cache_head / 8);
  const uint4 *vc = static_cast<const uint4 *>(a.d_v_cache) + h * (a.cache_head / 8);
  const T *kn = static_cast<const T *>(a.d_k_new) + b * a.k_new_batch + h * a.k_new_head;
  const T *vn = static_cast<const T *>(a.d_v_new) + b * a.v_new_batch + h * a.v_new_head;
  const uint32_t page_units = (uint32_t)(a.cache_page / 8), token_units = (uint32_t)(a.cache_token / 8);

  // Offsets, in 16-byte units, of the rows of key lane % 32 of a strip; keys
  // past the end stand for the last one.
  auto entry_of = [&](uint32_t strip) -> int32_t {
    if (strip >= q.strips_ctx) return 0;
    return q.table[k.page.quot(min(strip * 32 + (lane & 31), q.len - 1))];
  };
  auto offsets_of = [&](uint32_t strip, int32_t e, uint32_t &ko, uint32_t &vo) {
    if (strip < q.strips_ctx) {
      const uint32_t key = min(strip * 32 + (lane & 31), q.len - 1), page = min((uint32_t)max(e, 0), a.n_pages - 1);
      ko = vo = page * page_units + (key - k.page.quot(key) * k.page.d) * token_units;
    } else {
      const uint32_t key = min((strip - q.strips_ctx) * 32 + (lane & 31), q.live - 1);
      ko = key * (uint32_t)(a.k_new_node / 8);
      vo = key * (uint32_t)(a.v_new_node / 8);
    }
  };
  auto load_k = [&](uint32_t strip, uint32_t off) {
    const uint4 *base = strip < q.strips_ctx ? kc : reinterpret_cast<const uint4 *>(kn);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint4 *p = base + (uint32_t)__shfl((int)off, 16 * t + l16);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t c = 4 * s + g4;
        if (EXACT) {
          kf[t][s] = p[c];
        } else {
          kf[t][s] = p[c * 8 < D ? c : 0];
          if (c * 8 >= D) kf[t][s] = make_uint4(0, 0, 0, 0);
        }
      }
    }
  };
  auto load_v = [&](uint32_t strip, uint32_t off) {
    const uint4 *base = strip < q.strips_ctx ? vc : reinterpret_cast<const uint4 *>(vn);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 *p = base + (uint32_t)__shfl((int)off, 16 * (j >> 2) + 4 * g4 + (j & 3));
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        uint32_t d = (n * 16 + l16) * C;
        if (!EXACT && d >= D) d = 0;   // values past the head: computed, never stored
        const uint32_t *w = reinterpret_cast<const uint32_t *>(reinterpret_cast<const T *>(p) + d);
        if constexpr (C == 8) {
          const uint4 t = *reinterpret_cast<const uint4 *>(w);
          vr[j][n][0] = t.x; vr[j][n][1] = t.y; vr[j][n][2] = t.z; vr[j][n][3] = t.w;
        } else {
          const uint2 t = *reinterpret_cast<const uint2 *>(w);
          vr[j][n][0] = t.x; vr[j][n][1] = t.y;
        }
      }
    }
  };

  uint32_t strip = lo + kw;
  if (strip < hi) {
    uint32_t ko, vo;
    offsets_of(strip, entry_of(strip), ko, vo);
    load_k(strip, ko);
    load_v(strip, vo);
    int32_t entry = strip + ways < hi ? entry_of(strip + ways) : 0;
    while (true) {
      const uint32_t next = strip + ways;
      const bool more = next < hi, tree = strip >= q.strips_ctx;
      const uint32_t first = (tree ? strip - q.strips_ctx : strip) * 32;
      const uint32_t valid = min((tree ? q.live : q.len) - first, 32u);
      if (more) offsets_of(next, entry, ko, vo);

      float p[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < KS; ++e) s = Half<T>::mfma(kf[t][e], qf[u][e], s);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[u][4 * t + e] = s[e];
        }
      if (more) {
        load_k(next, ko);
        entry = next + ways < hi ? entry_of(next + ways) : 0;
      }

      // a last strip that is not full, and the tree's: keys that a row may not
      // see score -infinity, values that are no keys' or (tree) not finite
      // become 0
      uint32_t seen[U];
      bool strange = false;
      const bool special = tree || valid < 32;
      if (special) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t bits = valid < 32 ? (1u << valid) - 1u : 0xFFFFFFFFu;
          if (tree) {
            if (!alive[u])
              bits = 0;
            else if (a.d_mask)
              bits &= reinterpret_cast<const uint32_t *>(a.d_mask)[((uint64_t)b * a.nodes + node[u]) * k.mask_words +
                                                                    first / 32];
            else
              bits &= node[u] >= first + 31 ? 0xFFFFFFFFu : node[u] < first ? 0u : (2u << (node[u] - first)) - 1u;
          }
          seen[u] = bits;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool is_key = 16 * (j >> 2) + 4 * g4 + (j & 3) < valid;
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int w = 0; w < C / 2; ++w) {
              uint32_t t = is_key ? vr[j][n][w] : 0u;
              constexpr uint32_t E = Half<T>::kExp;
              if (tree && (t & E) == E) t &= 0xFFFF0000u, strange = true;
              if (tree && (t & (E << 16)) == (E << 16)) t &= 0x0000FFFFu, strange = true;
              vr[j][n][w] = t;
            }
        }
      }

      uint4 pf[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float top = kLowest;
#pragma unroll
        for (int j = 0; j < 8; ++j) p[u][j] *= a.scale;
        if (special) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = -__builtin_inff();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, p[u][j]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(top > m[u] + (kSlack + Half<T>::kLift))) {
          const float up = fmaxf(top - Half<T>::kLift, m[u]), shrink = exp_of(m[u] - up);
          m[u] = up;
          l[u] *= shrink;
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int f = 0; f < C; ++f) o[u][n][f] *= shrink;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[u][j] = exp_of(p[u][j] - m[u]);
          l[u] += p[u][j];
        }
        pf[u] = make_uint4(pack2<T>(p[u][0], p[u][1]), pack2<T>(p[u][2], p[u][3]), pack2<T>(p[u][4], p[u][5]),
                           pack2<T>(p[u][6], p[u][7]));
      }
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int f = 0; f < C; ++f) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = __builtin_amdgcn_perm(vr[2 * e + 1][n][f >> 1], vr[2 * e][n][f >> 1],
                                         f & 1 ? 0x07060302u : 0x05040100u);
          const uint4 vf = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int u = 0; u < U; ++u) o[u][n][f] = Half<T>::mfma(vf, pf[u], o[u][n][f]);
        }

      // Infinities and NaN among the tree's values: add them to the rows that
      // see them (each wave's p through its own part of `joint`).
      if (special && __any(strange)) {
        float *mine = joint + wave * (U * 8 * 64);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) mine[(u * 8 + j) * 64 + lane] = p[u][j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        for (uint32_t key = 0; key < valid; ++key) {
          const T *row = vn + (uint64_t)(first + key) * a.v_new_node;
          const uint32_t at = ((key >> 4) * 4 + (key & 3)) * 64 + ((key >> 2) & 3) * 16 + l16;
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int f = 0; f < C; ++f) {
                const uint32_t d = (n * 16 + 4 * g4 + i) * C + f;
                const float v = EXACT || d < D ? (float)row[d] : 0.f;
                if (!__builtin_isfinite(v)) {
#pragma unroll
                  for (int u = 0; u < U; ++u)
                    if (seen[u] >> key & 1u) o[u][n][f][i] += mine[u * 8 * 64 + at] * v;
                }
              }
        }
        __builtin_amdgcn_wave_barrier();
      }
      if (!more) break;
      load_v(next, vo);
      strip = next;
    }
  }

  // ---- join the waves that hold the same rows
#pragma unroll
  for (int u = 0; u < U; ++u) {
    l[u] += __shfl_xor(l[u], 16);
    l[u] += __shfl_xor(l[u], 32);
  }
  __syncthreads();
  for (uint32_t st = ways / 2; st; st >>= 1) {
    const uint32_t slot = (kw & (st - 1)) * row_ways + rw;
    float *mine = joint + slot * (NREG + 2 * U) * 64 + lane;
    if (kw >= st && kw < 2 * st) {
      uint32_t at = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        mine[64 * at++] = m[u];
        mine[64 * at++] = l[u];
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int f = 0; f < C; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[64 * at++] = o[u][n][f][e];
      }
    }
    __syncthreads();
    if (kw < st) {
      uint32_t at = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float m2 = mine[64 * at++], l2 = mine[64 * at++];
        const float up = fmaxf(m[u], m2);
        const float w1 = exp_of(m[u] - up), w2 = exp_of(m2 - up);
        m[u] = up;
        l[u] = l[u] * w1 + l2 * w2;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int f = 0; f < C; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[u][n][f][e] = o[u][n][f][e] * w1 + mine[64 * at++] * w2;
      }
    }
    __syncthreads();
  }
  if (kw != 0) return;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = row0 + 16 * u;
    if (r >= k.rows) continue;
    if (k.splits == 1) {
      const uint32_t head = h * k.group.d + (r - node[u] * k.group.d);
      T *dst = static_cast<T *>(a.d_out) + b * a.out_batch + node[u] * a.out_node + head * a.out_head;
      const bool any = alive[u] && l[u] != 0.f;
      const float inv = any ? 1.0f / l[u] : 0.f;
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t d = (n * 16 + 4 * g4 + e) * C;
          if (!EXACT && d >= D) continue;
          uint32_t w[C / 2];
#pragma unroll
          for (int f = 0; f < C; f += 2)
            w[f / 2] = any ? pack2<T>(o[u][n][f][e] * inv, o[u][n][f + 1][e] * inv) : 0u;
          if constexpr (C == 8)
            *reinterpret_cast<uint4 *>(dst + d) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2 *>(dst + d) = make_uint2(w[0], w[1]);
        }
      if (a.d_lse && g4 == 0)
        a.d_lse[((uint64_t)b * a.nodes + node[u]) * a.q_heads + head] =
            any ? m[u] + __log2f(l[u]) * kLn2 : -__builtin_inff();
    } else {
      const uint64_t at = (((uint64_t)b * a.kv_heads + h) * k.splits + split) * k.rows + r;
      if (g4 == 0) {
        k.part_ml[2 * at] = m[u];
        k.part_ml[2 * at + 1] = l[u];
      }
      float *dst = k.part + at * D;
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t d = (n * 16 + 4 * g4 + e) * C;
          if (!EXACT && d >= D) continue;
#pragma unroll
          for (int f = 0; f < C; f += 4)
            *reinterpret_cast<f32x4 *>(dst + d + f) =
                f32x4{o[u][n][f][e], o[u][n][f + 1][e], o[u][n][f + 2][e], o[u][n][f + 3][e]};
        }
    }
  }
}

// One wave per query row: the parts' sums, brought to their common maximum
// and added in the order of the splits (64 / LD of them side by side).
template <typename T, uint32_t LD>
__global__ __launch_bounds__(256) void k_tree_attention_join(TreeAttnArgs k, uint32_t ways) {
  const enc_tree_attention_args &a = k.a;
  constexpr uint32_t W = 64 / LD;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t item = blockIdx.x * kWavesA + (threadIdx.x >> 6);
  if (item >= a.batch * a.kv_heads * k.rows) return;
  const uint32_t bh = item / k.rows, r = item - bh * k.rows;
  const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
  const Seq q = sequence_of(a, b);
  const uint32_t chunk = split_chunk(q.strips, k.splits, ways);
  const uint32_t live = (q.strips + chunk - 1) / chunk;
  const uint32_t node = k.group.quot(r), head = h * k.group.d + (r - node * k.group.d);

  const uint64_t row = (uint64_t)bh * k.splits * k.rows + r;
  float m = kLowest;
  for (uint32_t s = lane; s < live; s += 64) m = fmaxf(m, k.part_ml[2 * (row + (uint64_t)s * k.rows)]);
  for (uint32_t o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  const uint32_t way = lane / LD, d = lane % LD * 4;
  float l = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (uint32_t s = way; s < live; s += W) {
    const uint64_t at = row + (uint64_t)s * k.rows;
    const float w = exp_of(k.part_ml[2 * at] - m);
    l += w * k.part_ml[2 * at + 1];
    if (d < a.head_dim) acc += *reinterpret_cast<const f32x4 *>(k.part + at * a.head_dim + d) * w;
  }
  for (uint32_t o = 32; o >= LD; o >>= 1) {
    l += __shfl_xor(l, o);
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], o);
  }
  const bool any = node < q.live && l != 0.f;
  const float inv = any ? 1.0f / l : 0.f;
  if (way == 0 && d < a.head_dim) {
    T *dst = static_cast<T *>(a.d_out) + b * a.out_batch + node * a.out_node + head * a.out_head + d;
    const uint2 w = any ? make_uint2(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv))
                        : make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(dst) = w;
  }
  if (a.d_lse && lane == 0)
    a.d_lse[((uint64_t)b * a.nodes + node) * a.q_heads + head] =
        any ? m + __log2f(l) * kLn2 : -__builtin_inff();
}

template <typename T, int DP, int U>
void launch_unit(const TreeAttnArgs &k, const TreeAttnPlan &p, hipStream_t s) {
  const uint32_t groups = k.a.batch * k.splits * k.a.kv_heads;
  const dim3 grid((groups + 7) / 8 * 8 * k.row_tiles), block(256);
  if (k.a.head_dim == DP)
    hipLaunchKernelGGL((k_tree_attention<T, DP, U, true>), grid, block, 0, s, k, p.row_ways);
  else
    hipLaunchKernelGGL((k_tree_attention<T, DP, U, false>), grid, block, 0, s, k, p.row_ways);
}

template <typename T, int DP>
void launch_dim(const TreeAttnArgs &k, const TreeAttnPlan &p, hipStream_t s) {
  if (p.units == 1)
    launch_unit<T, DP, 1>(k, p, s);
  else if (p.units == 2)
    launch_unit<T, DP, 2>(k, p, s);
  else if constexpr (DP <= 128)
    launch_unit<T, DP, 4>(k, p, s);
}

template <typename T>
void launch_type(const TreeAttnArgs &k, const TreeAttnPlan &p, hipStream_t s) {
  const uint32_t D = k.a.head_dim;
  if (D <= 64)
    launch_dim<T, 64>(k, p, s);
  else if (D <= 128)
    launch_dim<T, 128>(k, p, s);
  else
    launch_dim<T, 256>(k, p, s);
  if (k.splits == 1) return;
  const uint32_t ways = kWavesA / p.row_ways;
  const dim3 grid((k.a.batch * k.a.kv_heads * k.rows + kWavesA - 1) / kWavesA), block(256);
  if (D <= 64)
    hipLaunchKernelGGL((k_tree_attention_join<T, 16>), grid, block, 0, s, k, ways);
  else if (D <= 128)
    hipLaunchKernelGGL((k_tree_attention_join<T, 32>), grid, block, 0, s, k, ways);
  else
    hipLaunchKernelGGL((k_tree_attention_join<T, 64>), grid, block, 0, s, k, ways);
}

}  // namespace

// Rows: 16, 32 or 64 of them to a wave (64 rows of 128 values are 64 + 128
// registers of Q and O a lane; of 256 values, 32 rows are), then 1, 2 or 4
// waves of different rows, then tiles. Splits: enough workgroups to fill 256
// compute units several times over, with at least a strip for every wave.
TreeAttnPlan plan_tree_attention(const enc_tree_attention_args &a) {
  TreeAttnPlan p;
  const uint32_t rows = a.nodes * (a.q_heads / a.kv_heads);
  const uint32_t most = a.head_dim > 128 ? 2 : 4;
  p.units = rows <= 16 ? 1 : rows <= 32 ? 2 : most;
  const uint32_t waves = (rows + 16 * p.units - 1) / (16 * p.units);
  p.row_ways = waves <= 1 ? 1 : waves <= 2 ? 2 : 4;
  p.row_tiles = (waves + p.row_ways - 1) / p.row_ways;
  const uint32_t ways = kWavesA / p.row_ways;
  const uint64_t strips = ((uint64_t)a.max_pages * a.page_size + 31) / 32 + (a.nodes + 31) / 32;
  const uint64_t tiles = (uint64_t)a.batch * a.kv_heads * p.row_tiles;
  uint64_t splits = (1024 + tiles - 1) / tiles;
  const uint64_t cap = (strips + ways - 1) / ways;
  if (splits > cap) splits = cap;
  if (splits > 128) splits = 128;
  p.splits = splits < 1 ? 1 : (uint32_t)splits;
  const uint64_t parts = p.splits == 1 ? 0 : (uint64_t)a.batch * a.kv_heads * p.splits * rows;
  p.part_bytes = align_up(4 * parts * a.head_dim, 256);
  p.ml_bytes = align_up(8 * parts, 256);
  return p;
}

hipError_t launch_tree_attention(const TreeAttnArgs &k, const TreeAttnPlan &p, hipStream_t s) {
  if (k.a.dtype == 1)
    launch_type<__bf16>(k, p, s);
  else
    launch_type<_Float16>(k, p, s);
  return hipGetLastError();
}

}  // namespace enc
