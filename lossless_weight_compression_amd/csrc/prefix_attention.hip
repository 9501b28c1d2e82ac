// prefix_attention.hip -- attention of sequences that share their first cached
// tokens (enc_prefix_attention), and how many they share (enc_cache_shared).
//
// o = sum_j e^(s_j - m) v_j / l is taken in two kinds of pieces. Over the shared
// tokens the query rows of all sequences of a group (sequences x nodes x heads
// of a KV head) are one matrix, so the shared keys and values are read once for
// all of them; over the rest, each sequence's own tokens and its tree, rows are
// the sequence's. Each piece leaves its rows' maxima, sums and unnormalised
// outputs in fp32, and a last kernel joins a row's pieces in their order.
//
// Both kinds run in one kernel, k_pieces: a workgroup takes a tile of rows, a KV
// head and a range of keys. Its four waves hold the same rows and take strips of
// 32 keys in turn, straight from memory into registers: no barrier in the loop,
// and a range's sums are joined through LDS before they are written, so that a
// range costs one set of partial sums, not four. S^T = K Q^T and O^T += V^T P^T
// as in tree_attention.hip: S^T leaves lane l with keys 4 (l / 16) + i of query
// row l % 16, which, rounded, are the P^T fragment of the second product; V is
// transposed in registers.
//
// Shared tokens are bound by the matrix unit and the exponentials, own ones by
// HBM. A wave with 64 rows (U = 4) reads a strip once for 64 rows.
#include "attention_math.h"
#include "group_math.h"
#include "step_common.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace enc {
namespace {

constexpr uint32_t kWays = 4;          // waves of a workgroup, on different strips
constexpr uint32_t kPlanThreads = 1024;

struct Seq {
  uint32_t len, live;
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
  return q;
}

// ---- the plan: groups, then pieces of about the same work

template <typename V> __device__ __forceinline__ V wave_scan(V v) {   // inclusive
  const uint32_t lane = threadIdx.x & 63;
  for (uint32_t o = 1; o < 64; o <<= 1) {
    const V w = __shfl_up(v, o);
    if (lane >= o) v += w;
  }
  return v;
}
// Inclusive scan over the workgroup, with the total.
template <typename V> __device__ __forceinline__ V group_scan(V v, V *side, V &total) {
  v = wave_scan(v);
  const uint32_t wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) side[wave] = v;
  __syncthreads();
  V before = 0;
  total = 0;
  for (uint32_t w = 0; w < kPlanThreads / 64; ++w) {
    if (w < wave) before += side[w];
    total += side[w];
  }
  return before + v;
}

// Group g is the batch entries from the greatest start up to g to the greatest up
// to g + 1: for ascending starts the starts themselves, for any others ranges
// that do not overlap.
__global__ __launch_bounds__(kPlanThreads) void k_prefix_plan(PrefixAttnArgs k) {
  const enc_tree_attention_args &a = k.a;
  typedef unsigned long long u64;
  __shared__ uint32_t side[kPlanThreads / 64], tops[kPlanThreads / 64];
  __shared__ u64 side64[kPlanThreads / 64];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t per = a.nodes * k.group.d;              // rows of a sequence

  for (uint32_t b = tid; b < a.batch; b += kPlanThreads) {
    k.first[b] = 0;
    k.group_of[b] = ~0u;
  }
  uint32_t floor_ = 0;   // greatest start so far
  for (uint32_t g0 = 0; g0 <= k.groups; g0 += kPlanThreads) {
    const uint32_t g = g0 + tid;
    uint32_t v = g <= k.groups ? (uint32_t)max(0, min(k.starts[g], (int32_t)a.batch)) : 0u;
    for (uint32_t o = 1; o < 64; o <<= 1) {
      const uint32_t w = __shfl_up(v, o);
      if (lane >= o) v = max(v, w);
    }
    __syncthreads();
    if (lane == 63) tops[wave] = v;
    __syncthreads();
    uint32_t before = floor_;
    for (uint32_t w = 0; w < kPlanThreads / 64; ++w) {
      if (w < wave) before = max(before, tops[w]);
      floor_ = max(floor_, tops[w]);
    }
    if (g <= k.groups) k.ends[g] = max(v, before);
  }
  __syncthreads();
  // a wave to a group: what it shares, at most its shortest member's length
  for (uint32_t g = wave; g < k.groups; g += kPlanThreads / 64) {
    const uint32_t from = k.ends[g], to = k.ends[g + 1];
    uint32_t shared = (uint32_t)max(k.shared[g], 0);
    for (uint32_t b = from + lane; b < to; b += 64) shared = min(shared, sequence_of(a, b).len);
    for (uint32_t o = 32; o; o >>= 1) shared = min(shared, (uint32_t)__shfl_xor((int)shared, o));
    if (to - from < 2) shared = 0;                        // nobody to share with
    for (uint32_t b = from + lane; b < to; b += 64) {
      k.first[b] = shared;
      k.group_of[b] = g;
    }
    if (lane == 0) k.common[g] = shared;
  }
  __syncthreads();

  // work: strips of all tiles of rows, a strip of many rows counting more
  u64 work = 0, total;
  for (uint32_t g = tid; g < k.groups; g += kPlanThreads) {
    const uint32_t tiles = ((k.ends[g + 1] - k.ends[g]) * per + k.tile - 1) / k.tile;
    work += (u64)tiles * ((k.common[g] + 31) / 32) * k.weight;
  }
  for (uint32_t b = tid; b < a.batch; b += kPlanThreads) {
    const Seq q = sequence_of(a, b);
    work += (u64)k.own_tiles * ((q.len - k.first[b] + 31) / 32 + (q.live + 31) / 32);
  }
  group_scan(work, side64, total);
  const u64 each = min((total + k.slots - 1) / k.slots, (u64)1 << 30);
  const uint32_t own_size = (uint32_t)max((each + kWays - 1) / kWays * kWays, (u64)k.least);
  const uint32_t size = (uint32_t)max((each + k.weight * kWays - 1) / (k.weight * kWays) * kWays, (u64)k.least);

  uint32_t slots = 0, sum;
  for (uint32_t g0 = 0; g0 < k.groups; g0 += kPlanThreads) {
    const uint32_t g = g0 + tid;
    uint32_t rows = 0, tiles = 0, units = 0, n = 0;
    if (g < k.groups) {
      rows = (k.ends[g + 1] - k.ends[g]) * per;
      tiles = (rows + k.tile - 1) / k.tile;
      units = (k.common[g] + 31) / 32;
      n = (units + size - 1) / size;
    }
    const uint32_t incl = group_scan(n * tiles, side, sum), base = slots + incl - n * tiles;
    if (g < k.groups) k.group_parts[g] = make_uint2(base, n);
    for (uint32_t i = 0; i < n * tiles; ++i) {
      const uint32_t part = i / tiles, tile = i - part * tiles;
      PrefixItem it;
      it.b = k.ends[g];
      it.row0 = tile * k.tile;
      it.rows = rows;
      it.first = 0;
      it.ctx = k.common[g];
      it.tree = 0;
      it.lo = part * size;
      it.hi = min(units, it.lo + size);
      k.items[base + i] = it;
    }
    slots += sum;
  }
  if (tid == 0) k.counts[0] = slots;
  uint32_t own = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const uint32_t b = b0 + tid;
    uint32_t units = 0, n = 0;
    PrefixItem it;
    if (b < a.batch) {
      const Seq q = sequence_of(a, b);
      it.b = b;
      it.rows = per;
      it.first = k.first[b];
      it.ctx = q.len - it.first;
      it.tree = q.live;
      units = (it.ctx + 31) / 32 + (it.tree + 31) / 32;
      n = max((units + own_size - 1) / own_size, 1u);
    }
    const uint32_t incl = group_scan(n * k.own_tiles, side, sum), base = own + incl - n * k.own_tiles;
    if (b < a.batch) k.own_parts[b] = make_uint2(base, n);
    for (uint32_t i = 0; i < n * k.own_tiles; ++i) {
      const uint32_t part = i / k.own_tiles;
      it.row0 = (i - part * k.own_tiles) * k.own_tile;
      it.lo = part * own_size;
      it.hi = min(units, it.lo + own_size);
      k.items[slots + base + i] = it;
    }
    own += sum;
  }
  if (tid == 0) k.counts[1] = slots + own;
}

// ---- a piece

// U: 16-row units of the tile. EXACT: head_dim is DP. OWN: the sequence's own
// tokens and its tree; else shared ones.
template <typename T, int DP, int U, bool EXACT, bool OWN>
__device__ __forceinline__ void piece(const PrefixAttnArgs &k, uint32_t item, uint32_t h, uint64_t at, float *joint) {
  constexpr int KS = DP / 32;                   // k steps of Q K^T
  constexpr int C = DP >= 128 ? 8 : DP / 16;    // consecutive values a lane transposes
  constexpr int NH = DP / (16 * C);             // groups of 16 C values
  constexpr int NREG = U * NH * C * 4;          // accumulators a lane holds
  const enc_tree_attention_args &a = k.a;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l16 = lane & 15, g4 = lane >> 4;
  const uint32_t D = a.head_dim;
  PrefixItem it;
  {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(k.items + item);   // the workgroup's: scalars
    it.b = __builtin_amdgcn_readfirstlane(w[0]);
    it.row0 = __builtin_amdgcn_readfirstlane(w[1]);
    it.rows = __builtin_amdgcn_readfirstlane(w[2]);
    it.first = __builtin_amdgcn_readfirstlane(w[3]);
    it.ctx = __builtin_amdgcn_readfirstlane(w[4]);
    it.tree = __builtin_amdgcn_readfirstlane(w[5]);
    it.lo = __builtin_amdgcn_readfirstlane(w[6]);
    it.hi = __builtin_amdgcn_readfirstlane(w[7]);
  }
  const uint32_t b0 = it.b, first = OWN ? it.first : 0, ctx = it.ctx;
  const int32_t *table;
  {
    const uint32_t s = a.d_seqs ? (uint32_t)a.d_seqs[b0] : b0;
    table = a.d_table + (uint64_t)(s < a.max_seqs ? s : 0) * a.max_pages;
  }
  const uint32_t strips_ctx = (ctx + 31) / 32, lo = it.lo, hi = it.hi;

  // ---- Q fragments: query row l % 16 of each unit, 8 values per k step. A row
  // is (sequence, node, head of the group).
  uint4 qf[U][KS];
  uint32_t node[U];
  bool alive[U];
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;   // -scale (-q).k
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = it.row0 + 16 * u + l16, rr = min(r, it.rows - 1);
    const uint32_t turn = k.group.quot(rr), member = OWN ? 0 : k.nodes.quot(turn);
    node[u] = turn - member * a.nodes;
    const uint32_t head = h * k.group.d + (rr - turn * k.group.d), b = b0 + member;
    alive[u] = r < it.rows && node[u] < (OWN ? it.tree : a.nodes);
    const T *p = static_cast<const T *>(a.d_q) + b * a.q_batch + node[u] * a.q_node + head * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t d = 32 * s + 8 * g4;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (alive[u] && (EXACT || d < D)) v = *reinterpret_cast<const uint4 *>(p + d);
      qf[u][s] = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
    }
  }

  f32x4 o[U][NH][C];
  float m[U], l[U];   // m: of q.k, before the scale
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = kLowest;
    l[u] = 0.f;
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int f = 0; f < C; ++f) o[u][x][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  uint4 kf[2][KS];
  uint32_t vr[8][NH][C / 2];
  const uint4 *kc = static_cast<const uint4 *>(a.d_k_cache) + h * (a.cache_head / 8);
  const uint4 *vc = static_cast<const uint4 *>(a.d_v_cache) + h * (a.cache_head / 8);
  const T *kn = static_cast<const T *>(a.d_k_new) + b0 * a.k_new_batch + h * a.k_new_head;
  const T *vn = static_cast<const T *>(a.d_v_new) + b0 * a.v_new_batch + h * a.v_new_head;
  const uint32_t page_units = (uint32_t)(a.cache_page / 8), token_units = (uint32_t)(a.cache_token / 8);

  // Offsets, in 16-byte units, of the rows of key lane % 32 of a strip; keys past
  // the end stand for the last one.
  auto entry_of = [&](uint32_t strip) -> int32_t {
    if (OWN && strip >= strips_ctx) return 0;
    return table[k.page.quot(first + min(strip * 32 + (lane & 31), ctx - 1))];
  };
  auto offsets_of = [&](uint32_t strip, int32_t e, uint32_t &ko, uint32_t &vo) {
    if (!OWN || strip < strips_ctx) {
      const uint32_t key = first + min(strip * 32 + (lane & 31), ctx - 1), page = min((uint32_t)max(e, 0), a.n_pages - 1);
      ko = vo = page * page_units + (key - k.page.quot(key) * k.page.d) * token_units;
    } else {
      const uint32_t key = min((strip - strips_ctx) * 32 + (lane & 31), it.tree - 1);
      ko = key * (uint32_t)(a.k_new_node / 8);
      vo = key * (uint32_t)(a.v_new_node / 8);
    }
  };
  auto load_k = [&](uint32_t strip, uint32_t off) {
    const uint4 *base = !OWN || strip < strips_ctx ? kc : reinterpret_cast<const uint4 *>(kn);
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
    const uint4 *base = !OWN || strip < strips_ctx ? vc : reinterpret_cast<const uint4 *>(vn);
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

  // Bit j: node i may see node first + j.
  auto tree_bits = [&](uint32_t i, uint32_t from) -> uint32_t {
    if (from >= it.tree) return 0;
    uint32_t bits = it.tree - from < 32 ? (1u << (it.tree - from)) - 1u : 0xFFFFFFFFu;
    const uint32_t *mask = reinterpret_cast<const uint32_t *>(a.d_mask);
    if (mask)
      bits &= mask[((uint64_t)b0 * a.nodes + i) * k.mask_words + from / 32];
    else
      bits &= i >= from + 31 ? 0xFFFFFFFFu : i < from ? 0u : (2u << (i - from)) - 1u;
    return bits;
  };

  // One strip, its K and V on the way into the registers. SPECIAL: a last strip
  // that is not full, and the tree's: keys that a row may not see weigh nothing,
  // values that are no keys' or (tree) not finite become 0. `after_k` and
  // `after_v` load the next strip's halves.
  bool strange = false;   // infinities or NaN were among the tree's values
  const float c2 = k.unit, slack = k.slack;
  auto compute = [&](auto special_, uint32_t strip, auto after_k, auto after_v) {
    constexpr bool SPECIAL = decltype(special_)::value;
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
    after_k();

    const bool tree = OWN && SPECIAL && strip >= strips_ctx;
    const uint32_t from = (tree ? strip - strips_ctx : strip) * 32;
    const uint32_t valid = SPECIAL ? min((tree ? it.tree : ctx) - from, 32u) : 32;
    uint32_t seen[U];
    if constexpr (SPECIAL) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t bits = valid < 32 ? (1u << valid) - 1u : 0xFFFFFFFFu;
        if (tree) bits = alive[u] ? tree_bits(node[u], from) : 0u;
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
      if constexpr (SPECIAL) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = -__builtin_inff();
      }
      float top = p[u][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, p[u][j]);
      top = rows_max(top);
      if (__any(top - m[u] > slack)) {
        // only the rows concerned: what a row gives does not depend on the others
        const float up = top - m[u] > slack ? top : m[u], shrink = __builtin_amdgcn_exp2f((m[u] - up) * c2);
        m[u] = up;
        l[u] *= shrink;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int f = 0; f < C; ++f) o[u][n][f] *= shrink;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // the difference first: exact where it matters, however large the scores
        p[u][j] = __builtin_amdgcn_exp2f(fmaf(p[u][j] - m[u], c2, Half<T>::kLift2));
        if constexpr (SPECIAL)   // -infinity times a scale of 0 is no number
          if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = 0.f;
      }
      l[u] += ((p[u][0] + p[u][1]) + (p[u][2] + p[u][3])) + ((p[u][4] + p[u][5]) + (p[u][6] + p[u][7]));
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
    after_v();
  };

  const uint32_t whole = min(hi, ctx / 32);     // strips of 32 cached keys
  uint32_t strip = lo + wave;
  uint32_t ko, vo;
  if (strip < whole) {
    offsets_of(strip, entry_of(strip), ko, vo);
    load_k(strip, ko);
    load_v(strip, vo);
    int32_t entry = strip + kWays < whole ? entry_of(strip + kWays) : 0;
    while (true) {
      const uint32_t next = strip + kWays;
      const bool more = next < whole;
      if (more) offsets_of(next, entry, ko, vo);
      compute(
          std::false_type{}, strip,
          [&] {
            if (!more) return;
            load_k(next, ko);
            entry = next + kWays < whole ? entry_of(next + kWays) : 0;
          },
          [&] {
            if (more) load_v(next, vo);
          });
      strip = next;
      if (!more) break;
    }
  }
  for (; strip < hi; strip += kWays) {
    offsets_of(strip, entry_of(strip), ko, vo);
    load_k(strip, ko);
    load_v(strip, vo);
    compute(std::true_type{}, strip, [] {}, [] {});
  }
  // Infinities and NaN went in as zeros, since 0 times them would reach rows
  // that do not see them: add them to the rows that do.
  if (OWN && __any(strange)) {
    for (strip = lo + wave; strip < hi; strip += kWays) {
      if (strip < strips_ctx) continue;
      const uint32_t from = (strip - strips_ctx) * 32;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t seen = alive[u] ? tree_bits(node[u], from) : 0u;
        for (uint32_t key = 0; key < 32 && from + key < it.tree; ++key) {
          const T *row = vn + (uint64_t)(from + key) * a.v_new_node;
          if (!(seen >> key & 1u)) continue;
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int f = 0; f < C; ++f) {
                const uint32_t d = (n * 16 + 4 * g4 + i) * C + f;
                const float v = EXACT || d < D ? (float)row[d] : 0.f;
                if (!__builtin_isfinite(v)) o[u][n][f][i] += v;
              }
        }
      }
    }
  }

  // ---- join the waves
#pragma unroll
  for (int u = 0; u < U; ++u) l[u] = rows_sum(l[u]);
  for (uint32_t st = kWays / 2; st; st >>= 1) {
    float *mine = joint + (wave & (st - 1)) * (NREG + 2 * U) * 64 + lane;
    if (wave >= st && wave < 2 * st) {
      uint32_t i = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        mine[64 * i++] = m[u];
        mine[64 * i++] = l[u];
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int f = 0; f < C; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[64 * i++] = o[u][n][f][e];
      }
    }
    __syncthreads();
    if (wave < st) {
      uint32_t i = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float m2 = mine[64 * i++], l2 = mine[64 * i++];
        const float up = fmaxf(m[u], m2);
        const float w1 = __builtin_amdgcn_exp2f((m[u] - up) * c2), w2 = __builtin_amdgcn_exp2f((m2 - up) * c2);
        m[u] = up;
        l[u] = l[u] * w1 + l2 * w2;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int f = 0; f < C; ++f)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[u][n][f][e] = o[u][n][f][e] * w1 + mine[64 * i++] * w2;
      }
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (it.row0 + 16 * u + l16 >= it.rows) continue;
    const uint64_t row = at + 16 * u + l16;
    if (g4 == 0) *reinterpret_cast<float2 *>(k.part_ml + 2 * row) = make_float2(m[u], l[u]);
    float *dst = k.part + row * D;
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

// UP, US: units of a tile of shared and of own tokens' rows.
template <typename T, int DP, int UP, int US, bool EXACT>
__global__ __launch_bounds__(256, (DP == 256 || UP * DP > 256 ? 1 : 2)) void k_pieces(PrefixAttnArgs k) {
  constexpr int U = UP > US ? UP : US;
  __shared__ float joint[2 * (U * DP / 4 + 2 * U) * 64];
  const uint32_t heads = k.a.kv_heads, item = blockIdx.x / heads, h = blockIdx.x - item * heads;
  const uint32_t shared = __builtin_amdgcn_readfirstlane(k.counts[0]);
  if (item >= __builtin_amdgcn_readfirstlane(k.counts[1])) return;
  if (item < shared)
    piece<T, DP, UP, EXACT, false>(k, item, h, ((uint64_t)item * heads + h) * (16 * UP), joint);
  else
    piece<T, DP, US, EXACT, true>(k, item, h, k.own_rows + ((uint64_t)(item - shared) * heads + h) * (16 * US), joint);
}

// ---- the join: a wave to a query row, its pieces in their order, 64 / LD of
// them side by side
template <typename T, uint32_t LD>
__global__ __launch_bounds__(256) void k_prefix_join(PrefixAttnArgs k) {
  const enc_tree_attention_args &a = k.a;
  constexpr uint32_t W = 64 / LD;
  const uint32_t lane = threadIdx.x & 63, row = blockIdx.x * 4 + (threadIdx.x >> 6);
  const uint32_t per = a.nodes * k.group.d;
  if (row >= a.batch * a.kv_heads * per) return;
  const uint32_t bh = row / per, r = row - bh * per;
  const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
  const uint32_t node = k.group.quot(r), head = h * k.group.d + (r - node * k.group.d);
  int32_t live = a.d_nodes ? a.d_nodes[b] : (int32_t)a.nodes;
  const uint32_t g = k.group_of[b];
  const uint2 own = k.own_parts[b];
  uint2 common = make_uint2(0, 0);
  uint64_t at = 0, step = 0;   // rows of the shared pieces
  if (g != ~0u) {
    common = k.group_parts[g];
    const uint32_t from = k.ends[g], tiles = ((k.ends[g + 1] - from) * per + k.tile - 1) / k.tile;
    const uint32_t gr = (b - from) * per + r, tile = gr / k.tile;
    at = ((uint64_t)(common.x + tile) * a.kv_heads + h) * k.tile + (gr - tile * k.tile);
    step = (uint64_t)tiles * a.kv_heads * k.tile;
  }
  const uint32_t own_tile = r / k.own_tile;
  const uint64_t own_at = k.own_rows + ((uint64_t)(own.x + own_tile) * a.kv_heads + h) * k.own_tile + (r - own_tile * k.own_tile);
  const uint64_t own_step = (uint64_t)k.own_tiles * a.kv_heads * k.own_tile;
  const uint32_t parts = common.y + own.y;
  const auto row_of = [&](uint32_t s) { return s < common.y ? at + s * step : own_at + (s - common.y) * own_step; };
  const float2 *ml = reinterpret_cast<const float2 *>(k.part_ml);
  float m = kLowest;
  for (uint32_t s = lane; s < parts; s += 64) m = fmaxf(m, ml[row_of(s)].x);
  for (uint32_t o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  const uint32_t d = lane % LD * 4;
  const float *sums = k.part + (d < a.head_dim ? d : 0);
  float l = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (uint32_t s = lane / LD; s < parts; s += W) {
    const uint64_t p = row_of(s);
    const float2 part = ml[p];
    const f32x4 o = *reinterpret_cast<const f32x4 *>(sums + p * a.head_dim);
    const float w = __builtin_amdgcn_exp2f(fmaxf(part.x - m, kLowest) * k.unit);
    l += w * part.y;
    acc += o * w;
  }
  for (uint32_t o = 32; o >= LD; o >>= 1) {
    l += __shfl_xor(l, o);
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], o);
  }
  const bool any = (int32_t)node < live && l != 0.f;
  const float inv = any ? 1.0f / l : 0.f;
  if (lane < LD && d < a.head_dim) {
    T *dst = static_cast<T *>(a.d_out) + b * a.out_batch + node * a.out_node + head * a.out_head + d;
    const uint2 w = any ? make_uint2(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv))
                        : make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(dst) = w;
  }
  if (a.d_lse && lane == 0)
    a.d_lse[((uint64_t)b * a.nodes + node) * a.q_heads + head] =
        any ? m * fabsf(a.scale) + (__log2f(l) - Half<T>::kLift2) * kLn2 : -__builtin_inff();
}

template <typename T, int DP, int UP, int US>
void launch_pieces(const PrefixAttnArgs &k, const PrefixAttnPlan &p, hipStream_t s) {
  const dim3 grid(p.items * k.a.kv_heads), block(256);
  if (k.a.head_dim == DP)
    hipLaunchKernelGGL((k_pieces<T, DP, UP, US, true>), grid, block, 0, s, k);
  else
    hipLaunchKernelGGL((k_pieces<T, DP, UP, US, false>), grid, block, 0, s, k);
}

template <typename T, int DP>
void launch_dim(const PrefixAttnArgs &k, const PrefixAttnPlan &p, hipStream_t s) {
  constexpr int UP = DP <= 128 ? 4 : 2;
  if (p.tile == 16)
    launch_pieces<T, DP, 1, 1>(k, p, s);
  else if (p.own_tile == 16)
    launch_pieces<T, DP, UP, 1>(k, p, s);
  else
    launch_pieces<T, DP, UP, UP>(k, p, s);
}

template <typename T>
void launch_type(const PrefixAttnArgs &k, const PrefixAttnPlan &p, hipStream_t s) {
  const uint32_t D = k.a.head_dim, rows = k.a.batch * k.a.nodes * k.a.q_heads;
  hipLaunchKernelGGL(k_prefix_plan, dim3(1), dim3(kPlanThreads), 0, s, k);
  if (D <= 64)
    launch_dim<T, 64>(k, p, s);
  else if (D <= 128)
    launch_dim<T, 128>(k, p, s);
  else
    launch_dim<T, 256>(k, p, s);
  const dim3 grid((rows + 3) / 4), block(256);
  if (D <= 64)
    hipLaunchKernelGGL((k_prefix_join<T, 16>), grid, block, 0, s, k);
  else if (D <= 128)
    hipLaunchKernelGGL((k_prefix_join<T, 32>), grid, block, 0, s, k);
  else
    hipLaunchKernelGGL((k_prefix_join<T, 64>), grid, block, 0, s, k);
}

// ---- how many leading tokens the sequences of a group have in common: table
// entries are compared column by column, up to the first that differs
__global__ __launch_bounds__(kPlanThreads) void k_cache_shared(enc_cache c, const int32_t *seqs, uint32_t batch,
                                                               const int32_t *starts, int32_t *shared) {
  __shared__ uint32_t bottom, least, differs;
  const uint32_t g = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) bottom = 0, least = differs = ~0u;
  __syncthreads();
  const auto clamped = [&](uint32_t i) { return (uint32_t)max(0, min(starts[i], (int32_t)batch)); };
  uint32_t from = 0;
  for (uint32_t i = tid; i <= g; i += kPlanThreads) from = max(from, clamped(i));
  atomicMax(&bottom, from);
  __syncthreads();
  from = bottom;
  const uint32_t to = max(from, clamped(g + 1));
  if (from == to) {
    if (tid == 0) shared[g] = 0;
    return;
  }
  const uint32_t room = c.max_pages * c.page_size;   // below 2^31: checked on the host
  uint32_t len = ~0u;
  for (uint32_t b = from + tid; b < to; b += kPlanThreads) {
    const uint32_t s = (uint32_t)seqs[b];
    len = min(len, s < c.max_seqs ? min((uint32_t)max(c.d_lens[s], 0), room) : 0u);
  }
  atomicMin(&least, len);
  __syncthreads();
  len = least;
  const uint32_t pages = (len + c.page_size - 1) / c.page_size;
  // (len is not 0 below: every sequence is one of the table)
  const int32_t *row0 = c.d_table + (uint64_t)(uint32_t)seqs[from] * c.max_pages;
  for (uint32_t p0 = 0; p0 < pages; p0 += kPlanThreads) {
    const uint32_t p = p0 + tid;
    if (p < pages) {
      const int32_t e = row0[p];
      bool alike = e >= 0;
#pragma unroll 8
      for (uint32_t b = from + 1; b < to; ++b) alike &= c.d_table[(uint64_t)(uint32_t)seqs[b] * c.max_pages + p] == e;
      if (!alike) atomicMin(&differs, p);
    }
    __syncthreads();
    if (differs != ~0u) break;
    __syncthreads();
  }
  if (tid == 0) shared[g] = (int32_t)min((uint64_t)min(differs, pages) * c.page_size, (uint64_t)len);
}

}  // namespace

// Tiles of 64 rows (32 for heads above 128 values) where a group has more than
// 16 on average, of 16 below; the same for a sequence's own rows.
PrefixAttnPlan plan_prefix_attention(const enc_tree_attention_args &a, uint32_t groups) {
  PrefixAttnPlan p;
  const uint32_t per = a.nodes * (a.q_heads / a.kv_heads), large = a.head_dim <= 128 ? 64 : 32;
  const uint64_t rows = (uint64_t)a.batch * per;
  p.tile = per > 16 || rows > 16ull * std::max(groups, 1u) ? large : 16;
  p.own_tile = per > 16 ? large : 16;
  p.own_tiles = (per + p.own_tile - 1) / p.own_tile;
  p.weight = 1;
  p.slots = std::max(512 / a.kv_heads, 1u);
  p.least = kWays;
  // pieces of `slots` equal shares of the work, and one more, a short one, for
  // every tile
  const uint64_t tiles = std::min<uint64_t>(rows / p.tile + groups, rows);
  p.most_shared = (uint32_t)(p.slots + tiles);
  p.most_own = (uint32_t)(p.slots + (uint64_t)a.batch * p.own_tiles);
  p.items = p.most_shared + (uint32_t)((uint64_t)a.batch * p.own_tiles);
  const uint64_t n = (uint64_t)p.most_shared * a.kv_heads * p.tile + (uint64_t)p.most_own * a.kv_heads * p.own_tile;
  p.part_bytes = align_up(4 * n * a.head_dim, 256);
  p.ml_bytes = align_up(8 * n, 256);
  p.item_bytes = align_up(sizeof(PrefixItem) * (uint64_t)p.items, 256);
  p.batch_bytes = align_up(4ull * a.batch, 256);
  p.group_bytes = align_up(4ull * (groups + 1), 256);
  return p;
}

hipError_t launch_prefix_attention(PrefixAttnArgs k, const PrefixAttnPlan &p, hipStream_t s) {
  k.unit = std::min(std::fabs(k.a.scale) * kLog2e, -kLowest);
  k.slack = std::min(kSlack2 / k.unit, -kLowest);
  if (k.a.dtype == 1)
    launch_type<__bf16>(k, p, s);
  else
    launch_type<_Float16>(k, p, s);
  return hipGetLastError();
}

hipError_t launch_cache_shared(const enc_cache &c, const int32_t *seqs, uint32_t batch, const int32_t *starts,
                               uint32_t groups, int32_t *shared, hipStream_t s) {
  hipLaunchKernelGGL(k_cache_shared, dim3(groups), dim3(kPlanThreads), 0, s, c, seqs, batch, starts, shared);
  return hipGetLastError();
}

}  // namespace enc
