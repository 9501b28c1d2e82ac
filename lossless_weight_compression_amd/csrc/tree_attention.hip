// tree_attention.hip -- attention of a tree's nodes over a paged cache and
// the tree itself (enc_tree_attention).
//
// One pass over the keys with a running maximum m and sum l per query row:
// o = sum_j e^(s_j - m) v_j / l, s_j = scale q.k_j. The query rows that share a
// KV head (nodes x heads of its group) are one matrix, so every key and value
// is read once for all of them: HBM traffic of the cache is the bound, until
// some 200 rows share a KV head.
//
// Both kernels compute S^T = K Q^T and O^T += V^T P^T with v_mfma 16x16x32 on
// strips of 32 keys. S^T leaves lane l with keys 4 (l / 16) + i of query row
// l % 16. The sum over keys in P V may run in any order, so key 16 t + 4 g + i
// is made contraction index 8 g + 4 t + i: these registers, rounded, are then
// the P^T fragment, with no exchange between lanes. m and l belong to the
// lane's own query row; rescaling needs no exchange either.
//  * k_tree_attention, rows up to 16 (up to 32 in large batches): a wave holds
//    all rows, and K and V go from memory straight into its registers.
//    K: lane l holds 8 consecutive values of key l % 16, so fragments are
//    loaded from the rows as they lie, 16 bytes a lane. V: lane l loads, of its
//    group's 8 keys, values (l % 16) C .. + C - 1 (C = 8 for 128 values: whole
//    rows per 16 lanes) and transposes them in registers, one byte permute per
//    output dword. Row m of V^T fragment f then stands for value m C + f, and
//    lane l's accumulators hold runs of C consecutive values of its row, stored
//    16 bytes at a time.
//  * k_tree_attention_wide, more rows: 4 or 8 waves hold different rows and
//    share the keys through LDS. Its maxima are of q.k, before the scale.
//
// The matrix unit takes P in the values' type. k_tree_attention, which waits
// for memory, gives it P in two, the rounding and the rounded rest, so that the
// result's own rounding is what is left (BF16, against 64 bits: 1.66e-3 of the
// result's norm, 2.2e-3 with the rounding alone; one node over 1021 tokens 11.8
// us, 11.4 without, 16384 21.8 and 21.4, 131072 116.6 and 116.4, 64 sequences
// the same; at most 5% more, 64 sequences of up to 2000 tokens with 28 rows of
// 80 values).
// In the wide kernel the second product would cost more than half as much again
// (64 nodes over 131072 tokens: 197 us, 306 with it): there P is rounded, an
// error of up to 2^-8 of each weight for BF16, like the result's rounding. Sums,
// m, l and o are fp32. A row's m only moves when a strip of its own scores exceeds
// it by more than 8 (a factor of 2^8, far inside fp32 and both 16-bit ranges),
// which makes rescaling rare.
//
// The work is cut into equal parts over all sequences (share_of), so that one
// long history fills the device as well as many short ones do; a second kernel
// joins the parts of a row in their order.
//
// Measured (BF16, 8 KV heads of 128 under 32 query heads; us on the device with
// the join): one sequence of 131072 tokens, pages of 64, one node: 117, 4.6 TB/s;
// 16384 tokens: 22; 1021, pages of 16: 11.8. 64 sequences of up to 8192 tokens
// with 8 nodes: 219 + 11, 4.8 TB/s, where a large copy reaches 4.9; pages of 32
// to 256 take 230 as well. 64 nodes over 131072 tokens (256 rows to a KV head):
// 185 to 220 with the clock, 620 to 740 TFLOP/s, where a large library matrix
// product reaches 1190: the vector unit (exponentials, maxima, packing) is busy
// 40% of the cycles, the matrix unit 37%, LDS 23%; without the loads it takes
// 183, the loads alone 107. So no unit is the bound there: two waves to a SIMD,
// behind one barrier a stage, do not cover each other's dependent steps.
#include "attention_math.h"
#include "group_math.h"
#include "step_common.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace enc {
namespace {

constexpr uint32_t kWavesA = 4;
constexpr float kFar = 65536.f;   // see the wide kernel

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

// The work of a call in units of `unit` keys (a history's units, then its
// tree's), cut into parts of the same number of units over all sequences: a
// short sequence has one part, a long one many. Which part is whose follows
// from the lengths, which only the device knows: a wave adds up the units of
// all sequences, 64 at a time, and derives the part size, then finds its part
// (or its sequence's parts) in the running number of parts.
struct Share {
  uint32_t b;              // sequence
  uint32_t first, parts;   // its first part's number, and how many it has
  uint32_t size;           // units in a part
  bool found;
};

__device__ __forceinline__ uint32_t units_of(const enc_tree_attention_args &a, uint32_t b, uint32_t unit) {
  if (b >= a.batch) return 0;
  const Seq q = sequence_of(a, b);
  return (q.len + unit - 1) / unit + (q.live + unit - 1) / unit;
}

__device__ __forceinline__ Share share_of(const TreeAttnArgs &k, uint32_t unit, uint32_t ways, uint32_t part) {
  const enc_tree_attention_args &a = k.a;
  const uint32_t lane = threadIdx.x & 63;
  auto size_of = [&](uint32_t total) {
    const uint32_t each = (uint32_t)(((uint64_t)total + k.parts - 1) >> 32) ? total : (total + k.parts - 1) / k.parts;
    return max((each + ways - 1) / ways * ways, k.least);
  };
  Share s;
  if (a.batch == 1) {
    const uint32_t u = units_of(a, 0, unit);
    s.size = size_of(u);
    s.b = s.first = 0;
    s.parts = max((u + s.size - 1) / s.size, 1u);
    s.found = part < s.parts;
    return s;
  }
  const uint32_t mine = units_of(a, lane, unit);
  uint32_t total = 0;   // fits: checked on the host for the longest sequences the table holds
  for (uint32_t b0 = 0; b0 < a.batch; b0 += 64)
    total += __builtin_amdgcn_readlane(wave_incl_scan(b0 ? units_of(a, b0 + lane, unit) : mine), 63);
  s.size = size_of(total);
  s.found = false;
  s.b = s.first = s.parts = 0;
  uint32_t before = 0;
  for (uint32_t b0 = 0; b0 < a.batch; b0 += 64) {
    const uint32_t u = b0 ? units_of(a, b0 + lane, unit) : mine;
    const uint32_t n = b0 + lane < a.batch ? max((u + s.size - 1) / s.size, 1u) : 0;
    const uint32_t incl = wave_incl_scan(n), from = before + incl - n;
    const uint64_t hit = __ballot(n && part >= from && part < from + n);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      s.b = b0 + at;
      s.first = __builtin_amdgcn_readlane(from, at);
      s.parts = __builtin_amdgcn_readlane(n, at);
      s.found = true;
      return s;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return s;
}

// For the join: which parts are a sequence's.
__device__ __forceinline__ void note_parts(const TreeAttnArgs &k, const Share &s, uint32_t part, bool one) {
  if (k.shares && one && part == s.first && threadIdx.x == 0) k.shares[s.b] = make_uint2(s.first, s.parts);
}

// The kernel's arguments, read again where they are used: kept in scalar
// registers from the start, those of the first and last steps push the main
// loop's own into spills (a vector instruction for each use).
typedef const __attribute__((address_space(4))) TreeAttnArgs *ArgsPtr;
__device__ __forceinline__ ArgsPtr args_again() {
  ArgsPtr p = (ArgsPtr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// Bit j: node i of tree b may see node first + j.
__device__ __forceinline__ uint32_t tree_bits(uint32_t b, uint32_t i, uint32_t first, uint32_t live) {
  if (first >= live) return 0;
  uint32_t bits = live - first < 32 ? (1u << (live - first)) - 1u : 0xFFFFFFFFu;
  const ArgsPtr k = args_again();
  const uint32_t *mask = reinterpret_cast<const uint32_t *>(k->a.d_mask);
  if (mask)
    bits &= mask[((uint64_t)b * k->a.nodes + i) * k->mask_words + first / 32];
  else
    bits &= i >= first + 31 ? 0xFFFFFFFFu : i < first ? 0u : (2u << (i - first)) - 1u;
  return bits;
}

// DP: head_dim rounded up to what the fragments hold; EXACT: equal to it.
// U: 16-row units of a wave. Three workgroups to a compute unit are asked for
// where they just fit (heads of 96, 32768 tokens: 32.6 us, 37.0 with two).
// HEADS: the four waves take four neighbouring KV heads of the same keys, so
// rows of the cache that lie together are read together (64 sequences of up to
// 8192 tokens: 230 us, 251 without); else they take different strips of one
// head, joined through LDS at the end, and U is 1.
template <typename T, int DP, int U, bool EXACT, bool HEADS>
__global__ __launch_bounds__(256, (DP == 256 ? 1 : DP == 128 && U == 1 ? 3 : 2)) void k_tree_attention(TreeAttnArgs k) {
  constexpr int KS = DP / 32;                   // k steps of Q K^T
  constexpr int C = DP >= 128 ? 8 : DP / 16;    // consecutive values a lane transposes
  constexpr int NH = DP / (16 * C);             // groups of 16 C values
  constexpr int NREG = U * NH * C * 4;          // accumulators a lane holds
  const enc_tree_attention_args &a = k.a;
  __shared__ float joint[HEADS ? 1 : 2 * (NREG + 2 * U) * 64];

  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l16 = lane & 15, g4 = lane >> 4;
  const uint32_t D = a.head_dim;

  // neighbouring workgroups (on different dies) differ in their head, and each
  // die sees all heads
  const uint32_t sets = HEADS ? a.kv_heads / kWavesA : a.kv_heads;
  const uint32_t part = blockIdx.x / sets, set = (blockIdx.x + part) % sets;
  const uint32_t h = HEADS ? set * kWavesA + wave : set;
  constexpr uint32_t ways = HEADS ? 1 : kWavesA;
  const Share sh = share_of(k, 32, ways, part);
  if (!sh.found) return;
  note_parts(k, sh, part, set == 0);
  const uint32_t b = sh.b, kw = HEADS ? 0 : wave;
  const Seq q = sequence_of(a, b);
  const uint32_t strips_ctx = (q.len + 31) / 32, strips = strips_ctx + (q.live + 31) / 32;
  const uint32_t lo = (part - sh.first) * sh.size, hi = min(lo + sh.size, strips);

  // ---- Q fragments: query row l % 16 of each unit, 8 values per k step
  const uint32_t row0 = l16;
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
    if (strip >= strips_ctx) return 0;
    return q.table[k.page.quot(min(strip * 32 + (lane & 31), q.len - 1))];
  };
  auto offsets_of = [&](uint32_t strip, int32_t e, uint32_t &ko, uint32_t &vo) {
    if (strip < strips_ctx) {
      const uint32_t key = min(strip * 32 + (lane & 31), q.len - 1), page = min((uint32_t)max(e, 0), a.n_pages - 1);
      ko = vo = page * page_units + (key - k.page.quot(key) * k.page.d) * token_units;
    } else {
      const uint32_t key = min((strip - strips_ctx) * 32 + (lane & 31), q.live - 1);
      ko = key * (uint32_t)(a.k_new_node / 8);
      vo = key * (uint32_t)(a.v_new_node / 8);
    }
  };
  auto load_k = [&](uint32_t strip, uint32_t off) {
    const uint4 *base = strip < strips_ctx ? kc : reinterpret_cast<const uint4 *>(kn);
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
    const uint4 *base = strip < strips_ctx ? vc : reinterpret_cast<const uint4 *>(vn);
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

  // One strip, its K and V on the way into the registers. SPECIAL: a last strip
  // that is not full, and the tree's: keys that a row may not see score
  // -infinity, values that are no keys' or (tree) not finite become 0. SPLIT: P
  // in two parts. `after_k` and `after_v` load the next strip's halves.
  bool strange = false;   // infinities or NaN were among the tree's values
  auto compute = [&](auto special_, auto split_, uint32_t strip, auto after_k, auto after_v) {
    constexpr bool SPECIAL = decltype(special_)::value, SPLIT = decltype(split_)::value;
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

    const bool tree = SPECIAL && strip >= strips_ctx;
    const uint32_t first = (tree ? strip - strips_ctx : strip) * 32;
    const uint32_t valid = SPECIAL ? min((tree ? q.live : q.len) - first, 32u) : 32;
    uint32_t seen[U];
    if constexpr (SPECIAL) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t bits = valid < 32 ? (1u << valid) - 1u : 0xFFFFFFFFu;
        if (tree) bits = alive[u] ? tree_bits(b, node[u], first, q.live) : 0u;
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

    uint4 pf[U], pl[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float top = kLowest;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[u][j] *= a.scale;
        if constexpr (SPECIAL)
          if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = -__builtin_inff();
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, p[u][j]);
      top = rows_max(top);
      if (__any(top > m[u] + (kSlack + Half<T>::kLift))) {
        // only the rows concerned: what a row gives does not depend on the others
        const float up = top > m[u] + (kSlack + Half<T>::kLift) ? top - Half<T>::kLift : m[u], shrink = exp_of(m[u] - up);
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
      uint32_t round[4], rest[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a0 = p[u][2 * j], a1 = p[u][2 * j + 1];
        round[j] = pack2<T>(a0, a1);
        if (SPLIT) rest[j] = pack2<T>(a0 - half_of<T>(round[j], 0), a1 - half_of<T>(round[j], 1));
      }
      pf[u] = make_uint4(round[0], round[1], round[2], round[3]);
      if (SPLIT) pl[u] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
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
        for (int u = 0; u < U; ++u) {
          o[u][n][f] = Half<T>::mfma(vf, pf[u], o[u][n][f]);
          if (SPLIT) o[u][n][f] = Half<T>::mfma(vf, pl[u], o[u][n][f]);
        }
      }

    after_v();
  };

  const uint32_t whole = min(hi, q.len / 32);     // strips of 32 cached keys
  auto pass = [&](auto split_) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = kLowest;
      l[u] = 0.f;
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int f = 0; f < C; ++f) o[u][x][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    uint32_t strip = lo + kw;
    uint32_t ko, vo;
    if (decltype(split_)::value && strip < whole) {
      offsets_of(strip, entry_of(strip), ko, vo);
      load_k(strip, ko);
      load_v(strip, vo);
      int32_t entry = strip + ways < whole ? entry_of(strip + ways) : 0;
      while (true) {
        const uint32_t next = strip + ways;
        const bool more = next < whole;
        if (more) offsets_of(next, entry, ko, vo);
        compute(
            std::false_type{}, split_, strip,
            [&] {
              if (!more) return;
              load_k(next, ko);
              entry = next + ways < whole ? entry_of(next + ways) : 0;
            },
            [&] {
              if (more) load_v(next, vo);
            });
        strip = next;
        if (!more) break;
      }
    }
    for (; strip < hi; strip += ways) {
      offsets_of(strip, entry_of(strip), ko, vo);
      load_k(strip, ko);
      load_v(strip, vo);
      compute(std::true_type{}, split_, strip, [] {}, [] {});
    }
  };
  // The rest of a weight may be 0 or below, and then no number, or the wrong
  // infinity, comes of an infinite cached value. Every row sees that: where no
  // row is finite, once more without the rest, the simple way (the loop above a
  // second time, never run, cost 2% of every call).
  pass(std::true_type{});
  bool lost = true;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float zero = 0.f;
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int f = 0; f < C; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) zero = fmaf(o[u][n][f][e], 0.f, zero);
    lost = lost && rows_sum(zero) != 0.f;
  }
  if (__all(lost)) pass(std::false_type{});
  // Infinities and NaN went in as zeros, since 0 times them would reach rows
  // that do not see them: add them to the rows that do.
  if (__any(strange)) {
    for (uint32_t strip = lo + kw; strip < hi; strip += ways) {
      if (strip < strips_ctx) continue;
      const uint32_t first = (strip - strips_ctx) * 32;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t seen = alive[u] ? tree_bits(b, node[u], first, q.live) : 0u;
        for (uint32_t key = 0; key < 32 && first + key < q.live; ++key) {
          const T *row = vn + (uint64_t)(first + key) * a.v_new_node;
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

  // ---- join the waves that hold the same rows
#pragma unroll
  for (int u = 0; u < U; ++u) l[u] = rows_sum(l[u]);
  if constexpr (!HEADS) {
  __syncthreads();
  for (uint32_t st = ways / 2; st; st >>= 1) {
    const uint32_t slot = kw & (st - 1);
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
  }
  if (kw != 0) return;
  const ArgsPtr g = args_again();
  const uint32_t group = g->group.d;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = row0 + 16 * u;
    if (r >= g->rows) continue;
    if (sh.parts == 1) {
      const uint32_t head = h * group + (r - node[u] * group);
      T *dst = static_cast<T *>(g->a.d_out) + b * g->a.out_batch + node[u] * g->a.out_node + head * g->a.out_head;
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
      if (g->a.d_lse && g4 == 0)
        g->a.d_lse[((uint64_t)b * g->a.nodes + node[u]) * g->a.q_heads + head] =
            any ? m[u] + __log2f(l[u]) * kLn2 : -__builtin_inff();
    } else {
      const uint64_t at = ((uint64_t)part * g->a.kv_heads + h) * g->rows + r;
      if (g4 == 0) {
        g->part_ml[2 * at] = m[u];
        g->part_ml[2 * at + 1] = l[u];
      }
      float *dst = g->part + at * D;
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

// ---- many rows: K and V through LDS
//
// W waves of U units each hold W U 16 different rows and go through the same
// keys, a stage of SK at a time. Heads up to 128 values: three stages lie in
// LDS (the one computed, the next, whose first K fragments are read early, and
// the one a slower wave may still be in), a fourth is on its way into
// registers. Above: two, for want of registers and LDS. Banks: a wave reads one 16-byte
// chunk of 16 rows of K at a time, in groups of lanes that mix neighbouring
// chunks, so chunk c of row r lies at c ^ k_turn(r); of V it reads 32 bytes of
// 8 rows, so rows lie 32 bytes further apart than they are long. V^T fragments
// come from ds_read_b64_tr: of 16 lanes, lane 4 j + c names values 4 c .. 4 c
// + 3 of key j, and lane i gets value i of the 4 keys.
template <int NCH>
__device__ __forceinline__ constexpr uint32_t k_turn(uint32_t r) {
  return NCH == 8 ? r >> 1 & 7 : r & 15;   // 16 rows (two to 256 bytes, for 8 chunks) on 16 places
}

// Keys in a stage: two strips, or one where two would leave a compute unit
// with a single workgroup of four waves.
constexpr int stage_keys(int dp, int waves) { return dp == 256 || (dp == 128 && waves == 4) ? 32 : 64; }

template <typename T, int DP, int U, int W>
__global__ __launch_bounds__(64 * W, 2) void k_tree_attention_wide(TreeAttnArgs k) {
  constexpr int KS = DP / 32, NF = DP / 16, NCH = DP / 8;
  constexpr int SK = stage_keys(DP, W);
  constexpr bool PIPE = DP <= 128;                 // registers for a strip's K and V fragments at once
  constexpr uint32_t NB = PIPE ? 3 : 2;            // stages in LDS
  constexpr int NT = 64 * W, NR = SK * NCH / NT;   // chunks of K (and of V) a thread brings in
  constexpr int PITCH = NCH + 2;                   // 16-byte chunks from row to row of V
  const enc_tree_attention_args &a = k.a;
  __shared__ __align__(16) uint4 ks[NB][SK * NCH], vs[NB][SK * PITCH];
  __shared__ uint32_t odd;

  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t l16 = lane & 15, g4 = lane >> 4;
  const uint32_t D = a.head_dim;
  // row tiles of one (part, head) differ in 8, so they meet in one compute die's
  // L2 (workgroups go to the 8 dies in turn)
  const uint32_t id8 = blockIdx.x >> 3;
  const uint32_t grp = id8 / k.row_tiles * 8 + (blockIdx.x & 7), rt = id8 % k.row_tiles;
  const uint32_t part = grp / a.kv_heads, h = (grp + part) % a.kv_heads;
  const Share sh = share_of(k, SK, 1, part);
  if (!sh.found) return;
  note_parts(k, sh, part, h == 0 && rt == 0);
  const uint32_t b = sh.b;
  const Seq q = sequence_of(a, b);
  const uint32_t ctx = (q.len + SK - 1) / SK, stages = ctx + (q.live + SK - 1) / SK;
  const uint32_t lo = (part - sh.first) * sh.size, hi = min(lo + sh.size, stages);

  const uint32_t row0 = (rt * W + wave) * (U * 16) + l16;
  const bool busy = (rt * W + wave) * (U * 16) < k.rows;   // this wave has rows
  uint4 qf[U][KS];
  uint32_t node[U];
  bool alive[U];
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;   // -scale (-q).k
  const float c2 = k.unit, slack = k.slack;
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
      uint4 v = make_uint4(0, 0, 0, 0);
      if (alive[u] && d < D) v = *reinterpret_cast<const uint4 *>(p + d);
      qf[u][s] = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
    }
  }
  // A key's weight is 2^(p c2 - mc), p = q.k: one fma, exact until it is
  // rounded, so that mc, the row's maximum mr times c2 (less the lift), may be
  // rounded as it likes. From kFar on the rounding of mc alone is no longer
  // small beside 1: there it is 2^((p - mr) c2), whose difference is exact where
  // it is small.
  f32x4 o[U][NF];
  float mr[U], mc[U], l[U];   // mr: -infinity until the row has seen a key
#pragma unroll
  for (int u = 0; u < U; ++u) {
    mr[u] = -__builtin_inff();
    mc[u] = kLowest;
    l[u] = 0.f;
#pragma unroll
    for (int f = 0; f < NF; ++f) o[u][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  bool far = false;   // some row of the wave has got there
  auto beyond = [&](int u) { return !(fabsf(mc[u]) < kFar); };   // this one (or it has seen nothing)

  // ---- bringing a stage in: thread's chunk i is chunk ch of row r0 + i kRowStep
  const uint32_t ch = tid % NCH, r0 = tid / NCH;
  constexpr uint32_t kRowStep = NT / NCH, kWaveRows = 64 / NCH;
  const bool chunk_live = ch * 8 < D;
  const T *kc = static_cast<const T *>(a.d_k_cache) + h * a.cache_head;
  const T *vc = static_cast<const T *>(a.d_v_cache) + h * a.cache_head;
  // Where a page holds whole groups of the rows that a wave loads at once, the
  // page, its table entry and its address are the wave's: scalar work, and a
  // constant offset for each lane. Otherwise, and for a last stage that is not
  // full, each lane finds its own row.
  const bool by_wave = k.page.d % kWaveRows == 0 && a.cache_token * kWaveRows < (1u << 30);
  const uint32_t wave_row = __builtin_amdgcn_readfirstlane(r0);
  const uint32_t lane_off = (uint32_t)(r0 - wave_row) * (uint32_t)a.cache_token + ch * 8;
  typedef const __attribute__((address_space(4))) int32_t *const_ptr;   // read through the scalar cache
  const const_ptr table = (const_ptr)(uintptr_t)q.table;
  uint4 kr[NR], vr[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
  int32_t entry[NR];
  auto whole = [&](uint32_t st) { return st < ctx && (st + 1) * SK <= q.len; };
  auto find = [&](uint32_t st) {
    if (by_wave && whole(st)) {
#pragma unroll
      for (int i = 0; i < NR; ++i)
        entry[i] = table[__builtin_amdgcn_readfirstlane(k.page.quot(st * SK + wave_row + i * kRowStep))];
    } else if (st < ctx) {
#pragma unroll
      for (int i = 0; i < NR; ++i) entry[i] = q.table[k.page.quot(min(st * SK + r0 + i * kRowStep, q.len - 1))];
    }
  };
  auto fetch = [&](uint32_t st) {
    if (by_wave && whole(st)) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const uint32_t key = st * SK + wave_row + i * kRowStep;
        const uint32_t page = __builtin_amdgcn_readfirstlane(min((uint32_t)max(entry[i], 0), a.n_pages - 1));
        const uint32_t in = __builtin_amdgcn_readfirstlane(key - k.page.quot(key) * k.page.d);
        const uint64_t at = page * a.cache_page + in * a.cache_token;
        if (chunk_live) {
          kr[i] = *reinterpret_cast<const uint4 *>(kc + at + lane_off);
          vr[i] = *reinterpret_cast<const uint4 *>(vc + at + lane_off);
        }
      }
      return;
    }
    const bool tree = st >= ctx;
    const uint32_t first = (tree ? st - ctx : st) * SK, end = tree ? q.live : q.len;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint32_t key = first + r0 + i * kRowStep;
      kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
      if (key < end && chunk_live) {
        if (tree) {
          const ArgsPtr g = args_again();
          const T *kn = static_cast<const T *>(g->a.d_k_new) + b * g->a.k_new_batch + h * g->a.k_new_head;
          const T *vn = static_cast<const T *>(g->a.d_v_new) + b * g->a.v_new_batch + h * g->a.v_new_head;
          kr[i] = *reinterpret_cast<const uint4 *>(kn + key * g->a.k_new_node + ch * 8);
          vr[i] = *reinterpret_cast<const uint4 *>(vn + key * g->a.v_new_node + ch * 8);
        } else {
          const uint32_t page = min((uint32_t)max(entry[i], 0), a.n_pages - 1);
          const uint64_t at = page * a.cache_page + (key - k.page.quot(key) * k.page.d) * a.cache_token + ch * 8;
          kr[i] = *reinterpret_cast<const uint4 *>(kc + at);
          vr[i] = *reinterpret_cast<const uint4 *>(vc + at);
        }
      }
    }
  };
  auto place = [&](uint32_t st, uint32_t buf) {
    if (st >= ctx) {   // the tree's values go in finite
      asm volatile("");   // a branch, not selects on every stage's way
      constexpr uint32_t E = Half<T>::kExp;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        uint32_t w[4] = {vr[i].x, vr[i].y, vr[i].z, vr[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((w[e] & E) == E) w[e] &= 0xFFFF0000u, bad = true;
          if ((w[e] & (E << 16)) == (E << 16)) w[e] &= 0x0000FFFFu, bad = true;
        }
        vr[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (bad) odd = 1;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint32_t r = r0 + i * kRowStep;
      ks[buf][r * NCH + (ch ^ k_turn<NCH>(r))] = kr[i];
      vs[buf][r * PITCH + ch] = vr[i];
    }
  };

  // New maxima where a strip exceeds the old ones, and what is summed so far
  // brought to them; other rows stay as they are, to the bit.
  auto grow = [&](const float (&top)[U]) {
    bool out = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float up = top[u] - mr[u] > slack ? top[u] : mr[u], at = fmaf(up, c2, -Half<T>::kLift2);
      const bool was = beyond(u), is = !(fabsf(at) < kFar);
      const float by = was ? is ? (mr[u] - up) * c2 : fmaf(mr[u], c2, -at) - Half<T>::kLift2
                           : is ? fmaf(-up, c2, mc[u]) + Half<T>::kLift2 : mc[u] - at;
      const float shrink = mr[u] > -__builtin_inff() ? __builtin_amdgcn_exp2f(by) : 0.f;
      mr[u] = up;
      mc[u] = fmaxf(at, kLowest);
      out = out || (is && up > -__builtin_inff());
      l[u] *= shrink;
#pragma unroll
      for (int f = 0; f < NF; ++f) o[u][f] *= shrink;
    }
    far = __any(out);
  };

  // ---- one strip of 32 keys of a stage
  auto compute = [&](auto special_, uint32_t st, uint32_t half, uint32_t buf) {
    constexpr bool SPECIAL = decltype(special_)::value;
    const uint4 *row = ks[buf] + (half * 32 + l16) * NCH;
    const char *vb = reinterpret_cast<const char *>(vs[buf] + (half * 32 + 4 * g4 + (l16 >> 2)) * PITCH) + (l16 & 3) * 8;
    float p[U][8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x4 s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        const uint4 kf = row[16 * t * NCH + ((4 * e + g4) ^ k_turn<NCH>(l16))];
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = Half<T>::mfma(kf, qf[u][e], s[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[u][4 * t + e] = s[u][e];
      if constexpr (!PIPE) __builtin_amdgcn_sched_barrier(0);   // half of K at a time: registers
    }

    const bool tree = SPECIAL && st >= ctx;
    const uint32_t first = (tree ? st - ctx : st) * SK + half * 32, end = tree ? q.live : q.len;
    uint32_t seen[U];
    if constexpr (SPECIAL) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t bits = end >= first + 32 ? 0xFFFFFFFFu : end <= first ? 0u : (1u << (end - first)) - 1u;
        if (tree) bits = alive[u] ? tree_bits(b, node[u], first, q.live) : 0u;
        seen[u] = bits;
      }
    }
    uint4 pf[U];
    float top[U];
    bool grown = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (SPECIAL) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = -__builtin_inff();
      }
      float t = p[u][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) t = fmaxf(t, p[u][j]);
      top[u] = rows_max(t);
      grown = grown || top[u] - mr[u] > slack;
    }
    if (__any(grown)) grow(top);
    if (far) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float less = beyond(u) ? fmaxf(mr[u], kLowest) : 0.f, off = beyond(u) ? -Half<T>::kLift2 : mc[u];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[u][j] = __builtin_amdgcn_exp2f(fmaf(p[u][j] - less, c2, -off));
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) p[u][j] = __builtin_amdgcn_exp2f(fmaf(p[u][j], c2, -mc[u]));
    }
    if constexpr (SPECIAL) {   // -infinity times a scale of 0 is no number
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      l[u] += ((p[u][0] + p[u][1]) + (p[u][2] + p[u][3])) + ((p[u][4] + p[u][5]) + (p[u][6] + p[u][7]));
      pf[u] = make_uint4(pack2<T>(p[u][0], p[u][1]), pack2<T>(p[u][2], p[u][3]), pack2<T>(p[u][4], p[u][5]),
                         pack2<T>(p[u][6], p[u][7]));
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint2 v0 = read_transposed(vb + 32 * f), v1 = read_transposed(vb + 16 * PITCH * 16 + 32 * f);
      const uint4 vf = make_uint4(v0.x, v0.y, v1.x, v1.y);
#pragma unroll
      for (int u = 0; u < U; ++u) o[u][f] = Half<T>::mfma(vf, pf[u], o[u][f]);
    }
  };

  // ---- whole strips, two in flight: while the exponentials of one are taken,
  // the products of the next with K run, and while its products with V run,
  // the next's maxima are taken
  float p[U][8], top[U];
  uint4 kf[2][KS];
  auto read_k = [&](uint32_t buf, uint32_t half) {
    const uint4 *row = ks[buf] + (half * 32 + l16) * NCH;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < KS; ++e) kf[t][e] = row[16 * t * NCH + ((4 * e + g4) ^ k_turn<NCH>(l16))];
  };
  auto maxima = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float t = p[u][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) t = fmaxf(t, p[u][j]);
      top[u] = rows_max(t);
    }
  };
  auto scores = [&](float (&x)[U][8]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x4 s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < KS; ++e)
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = Half<T>::mfma(kf[t][e], qf[u][e], s[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[u][4 * t + e] = s[u][e];
    }
  };
  // (k_buf, k_half): the strip whose K is read here: the next one, before its
  // products, or, where a stage holds two strips, the one after it, as soon as
  // the next one's products have been started
  auto step = [&](uint32_t buf, uint32_t half, uint32_t k_buf, uint32_t k_half) {
    if constexpr (SK == 32) read_k(k_buf, k_half);
    uint4 vf[NF];
    const char *vb = reinterpret_cast<const char *>(vs[buf] + (half * 32 + 4 * g4 + (l16 >> 2)) * PITCH) + (l16 & 3) * 8;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint2 v0 = read_transposed(vb + 32 * f), v1 = read_transposed(vb + 16 * PITCH * 16 + 32 * f);
      vf[f] = make_uint4(v0.x, v0.y, v1.x, v1.y);
    }
    bool grown = false;
#pragma unroll
    for (int u = 0; u < U; ++u) grown = grown || top[u] - mr[u] > slack;
    if (__any(grown)) grow(top);
    float off[U];
#pragma unroll
    for (int u = 0; u < U; ++u) off[u] = mc[u];
    if (far) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float less = beyond(u) ? fmaxf(mr[u], kLowest) : 0.f;
        if (beyond(u)) off[u] = -Half<T>::kLift2;
#pragma unroll
        for (int j = 0; j < 8; ++j) p[u][j] -= less;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    float x[U][8];
    uint4 pf[U];
    scores(x);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[u][j] = __builtin_amdgcn_exp2f(fmaf(p[u][j], c2, -off[u]));
      l[u] += ((p[u][0] + p[u][1]) + (p[u][2] + p[u][3])) + ((p[u][4] + p[u][5]) + (p[u][6] + p[u][7]));
      pf[u] = make_uint4(pack2<T>(p[u][0], p[u][1]), pack2<T>(p[u][2], p[u][3]), pack2<T>(p[u][4], p[u][5]),
                         pack2<T>(p[u][6], p[u][7]));
    }
#pragma unroll
    for (int i = 0; i < 2 * KS * U; ++i) {   // a product, then a few of the others, in turn
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (SK == 64) {
      read_k(k_buf, k_half);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) p[u][j] = x[u][j];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int u = 0; u < U; ++u) o[u][f] = Half<T>::mfma(vf[f], pf[u], o[u][f]);
    maxima();
#pragma unroll
    for (int i = 0; i < NF * U; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  if (tid == 0) odd = 0;
  __syncthreads();
  if (lo < hi) {
    // one stage is placed ahead of the one that is computed (its first K is
    // read before the other's end), the one after it is on its way
    uint32_t st = lo, buf = 0;
    auto advance = [&] {
      const uint32_t next = buf + 1 == NB ? 0 : buf + 1;
      if constexpr (PIPE) {
        if (st + 1 < hi) place(st + 1, next);
        if (st + 2 < hi) fetch(st + 2);
        if (st + 3 < hi) find(st + 3);
      } else {
        place(st, buf);
        if (st + 1 < hi) fetch(st + 1);
        if (st + 2 < hi) find(st + 2);
      }
      __syncthreads();
      return next;
    };
    find(lo);
    fetch(lo);
    if (lo + 1 < hi) find(lo + 1);
    if constexpr (PIPE) {
      place(lo, 0);
      if (lo + 1 < hi) fetch(lo + 1);
      if (lo + 2 < hi) find(lo + 2);
    }
    const uint32_t whole_end = min(hi, q.len / SK);
    if constexpr (PIPE) {
      for (; st < whole_end; ++st) {
        const uint32_t next = advance();
        if (busy) {
          if (st == lo) {
            read_k(buf, 0);
            scores(p);
            maxima();
            if constexpr (SK == 64) read_k(buf, 1);
          }
          const bool more = st + 1 < whole_end;   // else: products that nobody asks for
          if constexpr (SK == 64) {
            step(buf, 0, more ? next : buf, 0);
            step(buf, 1, more ? next : buf, 1);
          } else {
            step(buf, 0, more ? next : buf, 0);
          }
        }
        buf = next;
      }
    }
    for (; st < hi; ++st) {
      const uint32_t next = advance();
      if (busy) {
        if (!PIPE && whole(st)) {
#pragma unroll 1
          for (uint32_t half = 0; half < SK / 32; ++half) compute(std::false_type{}, st, half, buf);
        } else {
#pragma unroll 1
          for (uint32_t half = 0; half < SK / 32; ++half) compute(std::true_type{}, st, half, buf);
        }
      }
      buf = next;
    }
  }
  if (!busy) return;
  const ArgsPtr g = args_again();
  const uint32_t group = g->group.d;
  // infinities and NaN, left out above: to the rows that see them
  if (hi > ctx && odd) {
    const T *vn = static_cast<const T *>(g->a.d_v_new) + b * g->a.v_new_batch + h * g->a.v_new_head;
#pragma unroll
    for (int u = 0; u < U; ++u)
      for (uint32_t first = (max(lo, ctx) - ctx) * SK; first < (hi - ctx) * SK && first < q.live; first += 32) {
        const uint32_t seen = alive[u] ? tree_bits(b, node[u], first, q.live) : 0u;
        for (uint32_t key = 0; key < 32 && first + key < q.live; ++key) {
          const T *row = vn + (uint64_t)(first + key) * g->a.v_new_node;
          if (!(seen >> key & 1u)) continue;
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t d = 16 * f + 4 * g4 + i;
              const float v = d < D ? (float)row[d] : 0.f;
              if (!__builtin_isfinite(v)) o[u][f][i] += v;
            }
        }
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    l[u] = rows_sum(l[u]);
    const uint32_t r = row0 + 16 * u;
    if (r >= g->rows) continue;
    // sums of weights 2^((p - mr) c2 + lift), whichever way they were taken
    const float fix = beyond(u) ? 1.f : __builtin_amdgcn_exp2f(fmaf(-mr[u], c2, mc[u]) + Half<T>::kLift2);
    if (sh.parts == 1) {
      const uint32_t head = h * group + (r - node[u] * group);
      T *dst = static_cast<T *>(g->a.d_out) + b * g->a.out_batch + node[u] * g->a.out_node + head * g->a.out_head;
      const bool any = alive[u] && l[u] != 0.f;
      const float inv = any ? 1.0f / l[u] : 0.f;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint32_t d = 16 * f + 4 * g4;
        if (d < D)
          *reinterpret_cast<uint2 *>(dst + d) =
              any ? make_uint2(pack2<T>(o[u][f][0] * inv, o[u][f][1] * inv), pack2<T>(o[u][f][2] * inv, o[u][f][3] * inv))
                  : make_uint2(0u, 0u);
      }
      if (g->a.d_lse && g4 == 0)
        g->a.d_lse[((uint64_t)b * g->a.nodes + node[u]) * g->a.q_heads + head] =
            any ? mr[u] * fabsf(g->a.scale) + (__log2f(l[u] * fix) - Half<T>::kLift2) * kLn2 : -__builtin_inff();
    } else {
      const uint64_t at = ((uint64_t)part * g->a.kv_heads + h) * g->rows + r;
      if (g4 == 0) {
        g->part_ml[2 * at] = fmaxf(mr[u], kLowest);
        g->part_ml[2 * at + 1] = l[u] * fix;
      }
      float *dst = g->part + at * D;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint32_t d = 16 * f + 4 * g4;
        if (d < D) *reinterpret_cast<f32x4 *>(dst + d) = o[u][f] * fix;
      }
    }
  }
}

// One query row to WAVES waves: the parts' sums, brought to their common
// maximum and added in a fixed order, WAVES 64 / LD of them side by side. The
// loads of a part do not depend on another's, so many are in flight.
template <typename T, uint32_t LD, uint32_t WAVES>
__global__ __launch_bounds__(256) void k_tree_attention_join(TreeAttnArgs k) {
  const enc_tree_attention_args &a = k.a;
  constexpr uint32_t W = WAVES * 64 / LD;
  __shared__ float side[WAVES == 1 ? 1 : 4 * 5 * 64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t item = WAVES == 1 ? blockIdx.x * kWavesA + wave : blockIdx.x;
  if (item >= a.batch * a.kv_heads * k.rows) return;
  const uint32_t bh = item / k.rows, r = item - bh * k.rows;
  const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
  const uint2 sh = k.shares[b];
  if (sh.y <= 1) return;   // written by its only part
  const Seq q = sequence_of(a, b);
  const uint32_t parts = sh.y;
  const uint32_t node = k.group.quot(r), head = h * k.group.d + (r - node * k.group.d);

  const uint64_t row = ((uint64_t)sh.x * a.kv_heads + h) * k.rows + r, step = (uint64_t)a.kv_heads * k.rows;
  const float2 *ml = reinterpret_cast<const float2 *>(k.part_ml) + row;
  float m = kLowest;
  for (uint32_t s = lane; s < parts; s += 64) m = fmaxf(m, ml[s * step].x);
  for (uint32_t o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  const uint32_t way = (WAVES == 1 ? 0 : wave * (64 / LD)) + lane / LD, d = lane % LD * 4;
  const float *sums = k.part + row * a.head_dim + (d < a.head_dim ? d : 0);
  float l = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (uint32_t s = way; s < parts; s += W) {
    const float2 part = ml[s * step];
    const f32x4 o = *reinterpret_cast<const f32x4 *>(sums + s * step * a.head_dim);
    const float w = __builtin_amdgcn_exp2f(fmaxf(part.x - m, kLowest) * k.unit);
    l += w * part.y;
    acc += o * w;
  }
  for (uint32_t o = 32; o >= LD; o >>= 1) {
    l += __shfl_xor(l, o);
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], o);
  }
  if constexpr (WAVES > 1) {
    float *mine = side + wave * 5 * 64 + lane;
    mine[0] = l;
    for (int e = 0; e < 4; ++e) mine[64 * (e + 1)] = acc[e];
    __syncthreads();
    if (wave != 0) return;
    for (uint32_t w = 1; w < WAVES; ++w) {
      l += side[w * 5 * 64 + lane];
      for (int e = 0; e < 4; ++e) acc[e] += side[w * 5 * 64 + 64 * (e + 1) + lane];
    }
  }
  const bool any = node < q.live && l != 0.f;
  const float inv = any ? 1.0f / l : 0.f;
  if (lane < LD && d < a.head_dim) {
    T *dst = static_cast<T *>(a.d_out) + b * a.out_batch + node * a.out_node + head * a.out_head + d;
    const uint2 w = any ? make_uint2(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv))
                        : make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(dst) = w;
  }
  if (a.d_lse && lane == 0)
    a.d_lse[((uint64_t)b * a.nodes + node) * a.q_heads + head] =
        any ? (k.raw ? m * fabsf(a.scale) - Half<T>::kLift : m) + __log2f(l) * kLn2 : -__builtin_inff();
}

template <typename T, int DP, int U>
void launch_unit(const TreeAttnArgs &k, const TreeAttnPlan &p, hipStream_t s) {
  const dim3 grid(k.grid_parts * (p.ways == 1 ? k.a.kv_heads / kWavesA : k.a.kv_heads)), block(256);
  if (p.ways == 1 && k.a.head_dim == DP)
    hipLaunchKernelGGL((k_tree_attention<T, DP, U, true, true>), grid, block, 0, s, k);
  else if (p.ways == 1)
    hipLaunchKernelGGL((k_tree_attention<T, DP, U, false, true>), grid, block, 0, s, k);
  else if constexpr (U == 1) {
    if (k.a.head_dim == DP)
      hipLaunchKernelGGL((k_tree_attention<T, DP, 1, true, false>), grid, block, 0, s, k);
    else
      hipLaunchKernelGGL((k_tree_attention<T, DP, 1, false, false>), grid, block, 0, s, k);
  }
}

template <typename T, int DP, int U, int W>
void launch_wide(const TreeAttnArgs &k, hipStream_t s) {
  const uint32_t groups = k.grid_parts * k.a.kv_heads;
  hipLaunchKernelGGL((k_tree_attention_wide<T, DP, U, W>), dim3((groups + 7) / 8 * 8 * k.row_tiles), dim3(64 * W), 0, s,
                     k);
}

template <typename T, int DP>
void launch_dim(const TreeAttnArgs &k, const TreeAttnPlan &p, hipStream_t s) {
  if (p.wide) {
    if (p.waves == 4 && p.units == 1) {
      launch_wide<T, DP, 1, 4>(k, s);
    } else if (p.waves == 4) {
      if constexpr (DP <= 128) launch_wide<T, DP, 2, 4>(k, s);
    } else if (p.units == 1) {
      launch_wide<T, DP, 1, 8>(k, s);
    } else if constexpr (DP <= 128) {
      launch_wide<T, DP, 2, 8>(k, s);
    }
  } else if (p.units == 1) {
    launch_unit<T, DP, 1>(k, p, s);
  } else if constexpr (DP <= 128) {
    launch_unit<T, DP, 2>(k, p, s);
  }
}

// Four waves to a row while the rows alone do not fill the device (131072
// tokens, one node: 117 us in all, 166 with one wave to a row).
template <typename T, uint32_t LD>
void launch_join(const TreeAttnArgs &k, hipStream_t s) {
  const uint32_t rows = k.a.batch * k.a.kv_heads * k.rows;
  if (rows <= 4096)
    hipLaunchKernelGGL((k_tree_attention_join<T, LD, 4>), dim3(rows), dim3(256), 0, s, k);
  else
    hipLaunchKernelGGL((k_tree_attention_join<T, LD, 1>), dim3((rows + kWavesA - 1) / kWavesA), dim3(256), 0, s, k);
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
  if (!p.part_bytes) return;
  if (D <= 64)
    launch_join<T, 16>(k, s);
  else if (D <= 128)
    launch_join<T, 32>(k, s);
  else
    launch_join<T, 64>(k, s);
}

}  // namespace

// Parts: as many as workgroups fit the device at once by their registers, with
// a stage (or a strip for every wave) each at least: 16384 tokens and one node
// took 50 us with 256 workgroups and 22 so; twice as many for the wide kernel
// were slower at 64 nodes over 131072 tokens.
TreeAttnPlan plan_tree_attention(const enc_tree_attention_args &a) {
  TreeAttnPlan p;
  const uint32_t rows = a.nodes * (a.q_heads / a.kv_heads);
  const uint64_t heads = (uint64_t)a.batch * a.kv_heads;
  const bool large = a.head_dim > 128;
  // Four heads to a workgroup where that leaves two waves to a compute unit
  // before any history is split. 8 nodes of 4 heads, 64 sequences of up to 8192
  // tokens: 228 us, in the wide kernel 264; 32 sequences of up to 4096: 87, wide
  // 84; one of 65536: 58, wide 52.
  const bool by_heads = a.kv_heads % 4 == 0 && heads >= 512;
  uint64_t fill;
  if (rows <= 16 || (rows <= 32 && !large && by_heads)) {
    p.wide = 0;
    p.units = rows <= 16 ? 1 : 2;
    p.waves = 4;
    p.ways = by_heads ? 1 : 4;
    p.unit = 32;
    p.row_tiles = 1;
    // workgroups that 256 compute units hold at once, by the registers of a wave
    fill = 256 * (a.head_dim <= 64 ? 5 - p.units : large ? 1 : 4 - p.units) * (4 / p.ways);
  } else {
    // Waves hold different rows, 16 or 32 each, 4 or 8 to a workgroup, then
    // tiles. With 32 a wave reads each fragment from LDS once for two products
    // (132 rows: 83 us against 154). 65 to 128 rows: four waves of 32 where
    // there are many sequences and heads (16 sequences of up to 4096 tokens, 100
    // rows: 56 us against 70 with eight of 16); eight of 16 where histories are
    // split more, whose parts are then half as many (1024 tokens: 13.5 against
    // 16.7; 65536: 72 against 77).
    p.wide = 1;
    const bool four = rows <= 64 || (rows <= 128 && !large && heads >= 128);
    p.units = large || rows <= 64 || (rows <= 128 && !four) ? 1 : 2;
    p.waves = four ? 4 : 8;
    p.ways = 1;
    p.unit = stage_keys(large ? 256 : a.head_dim > 64 ? 128 : 64, p.waves);
    const uint32_t tile = 16 * p.units * p.waves;
    p.row_tiles = (rows + tile - 1) / tile;
    fill = p.waves == 4 ? 512 : 256;
  }
  // at most `parts` equal parts, and one more for each sequence (its last, short
  // one); where that is a small share, they count towards the fill
  const uint64_t tiles = (uint64_t)a.kv_heads * p.row_tiles;
  const uint64_t units = ((uint64_t)a.max_pages * a.page_size + p.unit - 1) / p.unit + (a.nodes + p.unit - 1) / p.unit;
  uint64_t want = (fill + tiles - 1) / tiles;
  want = want >= 2ull * a.batch ? want - a.batch : want;
  const uint64_t most = (units + p.ways - 1) / p.ways * a.batch;
  p.parts = (uint32_t)(want < most ? want : most);
  p.grid_parts = p.parts + a.batch;
  // a part is at least a round of the ways; where no history is longer than
  // three rounds, one part without a join is quicker (300 tokens, 32 sequences:
  // 11.5 against 15.2 us; at 1000 tokens the join wins, 10.7 against 18.7)
  p.least = units <= 3 * p.ways ? 3 * p.ways : p.ways;
  const uint64_t parts = units <= p.least ? 0 : (uint64_t)p.grid_parts * a.kv_heads * rows;
  p.part_bytes = align_up(4 * parts * a.head_dim, 256);
  p.ml_bytes = align_up(8 * parts, 256);
  p.share_bytes = parts ? align_up(8ull * a.batch, 256) : 0;
  return p;
}

hipError_t launch_tree_attention(TreeAttnArgs k, const TreeAttnPlan &p, hipStream_t s) {
  k.raw = p.wide;
  k.unit = p.wide ? std::min(std::fabs(k.a.scale) * kLog2e, -kLowest) : kLog2e;
  k.slack = std::min(kSlack2 / k.unit, -kLowest);
  if (k.a.dtype == 1)
    launch_type<__bf16>(k, p, s);
  else
    launch_type<_Float16>(k, p, s);
  return hipGetLastError();
}

}  // namespace enc
