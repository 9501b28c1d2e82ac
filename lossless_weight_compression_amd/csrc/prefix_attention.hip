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
// S^T = K Q^T and O^T += V^T P^T as in tree_attention.hip: S^T leaves lane l with
// keys 4 (l / 16) + i of query row l % 16, which, rounded, are the P^T fragment of
// the second product. Which pieces there are the device finds from the lengths:
// k_prefix_plan* cut shared and own work into equal shares.
//
// The matrix unit takes P in the values' type: it gets the rounding and the rounded
// rest, two products, so that the result's own rounding is what is left. Before
// the rest, 4 sequences over 1021 tokens took 16.1 us (16.3 with it), 64 over 8192
// with 512 own tokens 63.0 (66.9), 16 over 131072 132.5 (133.1); 256 rows over
// 131072 tokens, which wait for the matrix unit, 214 (263).
//
// k_shared, groups of many rows: eight waves to a workgroup, 64 or 128 rows, a KV
// head and a range of keys. Keys and values go through LDS in stages of 64, used
// by four tiles of rows each; two waves to a tile take half of a stage's keys
// each. Two stages are on their way in registers, three lie in LDS (with one on
// its way times are within 2%, 131072 tokens either way 132 us a call). Long ranges
// of many rows run at 560 TFLOP/s of the formula's operations, 840 with the rests'
// (256 rows, from 8192 to 32768 tokens; some 4000 cycles a stage of 64 keys): the
// vector unit is busy 48% of the cycles, with the exponentials and conversions, the
// matrix unit 34%, LDS 20%; a piece's start and end, some 10 us, is the rest of a
// short call. Few rows are bound by HBM: 64 rows, 131072 tokens of 8 heads, 103 us =
// 5.2 TB/s.
//
// k_pieces, each sequence's own tokens and tree, and groups of few rows: four
// waves hold the same rows and take strips of 32 keys in turn, straight from
// memory into registers, with no barrier in the loop; V is transposed in
// registers; the waves' sums are joined through LDS before they are written, so
// that a range costs one set of partial sums, not four. It is bound by HBM, and in
// short calls by the way from the table to the keys. (For the shared tokens of
// many rows it took 33 us with 32 rows to a wave and 45 with 64, k_shared 24, all
// without the rests.)
//
// Measured, BF16, heads of 128, 32 query and 8 KV heads, whole call on the device:
// 4 sequences over 1021 shared tokens 16.2 us (plan 6.1, pieces 7.2, join 4.7); 64
// over 8192 with 512 own tokens at most 66.9 (6.1, shared 26.7, own 22.2, join 6.7;
// 5.2 for enc_cache_shared); 16 over 131072 133 (6.1, 103, 15.4, 8.0). Heads of 256:
// 16 over 8192 with 300 own 53.
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
  uint32_t len, live, row;   // row: of the table
};

__device__ __forceinline__ Seq sequence_of(const enc_tree_attention_args &a, uint32_t b) {
  Seq q;
  const uint32_t s = a.d_seqs ? (uint32_t)a.d_seqs[b] : b;
  const uint64_t room = (uint64_t)a.max_pages * a.page_size;
  int32_t len = s < a.max_seqs ? a.d_lens[s] : 0;
  len = max(len, 0);
  q.len = (uint64_t)len > room ? (uint32_t)room : (uint32_t)len;
  q.row = s < a.max_seqs ? s : 0;
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

// Strips in a piece: an equal share of all, whole rounds of the waves.
__device__ __forceinline__ uint32_t size_of(unsigned long long work, uint32_t slots, uint32_t least) {
  const unsigned long long each = min((work + slots - 1) / slots, 1ull << 30);
  return (uint32_t)max((each + kWays - 1) / kWays * kWays, (unsigned long long)least);
}

// The plan where every group and every sequence has a thread: numbers stay in
// registers and LDS, and the loads that they come from are on their way at once
// (one group of 64 sequences: 5.9 us, 12 by the general kernel below). Group g is the batch
// entries from the greatest start up to g to the greatest up to g + 1: for
// ascending starts the starts themselves, for any others ranges that do not
// overlap.
__global__ __launch_bounds__(kPlanThreads) void k_prefix_plan_small(PrefixAttnArgs k) {
  const enc_tree_attention_args &a = k.a;
  typedef unsigned long long u64;
  __shared__ uint32_t ends[kPlanThreads + 1], common[kPlanThreads], group_at[kPlanThreads + 1], own_at[kPlanThreads + 1];
  __shared__ uint32_t first[kPlanThreads], lens[kPlanThreads], lives[kPlanThreads], seqs[kPlanThreads];
  __shared__ uint32_t tops[kPlanThreads / 64];
  __shared__ u64 side[kPlanThreads / 64], side2[kPlanThreads / 64], side3[kPlanThreads / 64];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;   // > groups, >= batch
  const uint32_t per = a.nodes * k.group.d, groups = k.groups, batch = a.batch;
  // (without groups there need be no starts)
  uint32_t v = groups && tid <= groups ? (uint32_t)max(0, min(k.starts[tid], (int32_t)batch)) : 0u;
  const uint32_t asked = tid < groups ? (uint32_t)max(k.shared[tid], 0) : 0u;
  Seq q;
  q.len = q.live = q.row = 0;
  if (tid < batch) q = sequence_of(a, tid);

  for (uint32_t o = 1; o < 64; o <<= 1) {
    const uint32_t w = __shfl_up(v, o);
    if (lane >= o) v = max(v, w);
  }
  if (lane == 63) tops[wave] = v;
  __syncthreads();
  for (uint32_t w = 0; w < wave; ++w) v = max(v, tops[w]);
  ends[tid] = v;   // past the last group: the last end, or greater ones that nobody reads
  if (tid < groups) common[tid] = asked;
  __syncthreads();
  // the group of this thread's sequence: the last one that begins at or before it
  uint32_t g = ~0u;
  if (tid < batch && groups && tid >= ends[0] && tid < ends[groups]) {
    uint32_t low = 0, high = groups;   // ends[low] <= tid < ends[high]
    while (high - low > 1) {
      const uint32_t mid = (low + high) / 2;
      if (ends[mid] <= tid) low = mid; else high = mid;
    }
    g = low;
    atomicMin(&common[g], q.len);
  }
  __syncthreads();
  uint32_t rows = 0, tiles = 0, units = 0;
  if (tid < groups) {
    const uint32_t n = ends[tid + 1] - ends[tid];
    if (n < 2) common[tid] = 0;   // nobody to share with
    rows = n * per;
    tiles = (rows + k.tile - 1) / k.tile;
    units = (common[tid] + 31) / 32;
  }
  __syncthreads();
  uint32_t own_units = 0;
  if (tid < batch) {
    const uint32_t f = g != ~0u ? common[g] : 0u;
    first[tid] = f;
    lens[tid] = q.len;
    lives[tid] = q.live;
    seqs[tid] = q.row;
    own_units = (q.len - f + 31) / 32 + (q.live + 31) / 32;
    k.group_of[tid] = g;
    k.first[tid] = f;
  }
  u64 work = (u64)tiles * units, own_work = (u64)k.own_tiles * own_units;
  for (uint32_t o = 32; o; o >>= 1) {
    work += __shfl_xor(work, o);
    own_work += __shfl_xor(own_work, o);
  }
  if (lane == 0) side[wave] = work, side2[wave] = own_work;
  __syncthreads();
  work = own_work = 0;
  for (uint32_t w = 0; w < threads / 64; ++w) work += side[w], own_work += side2[w];
  const uint32_t size = size_of(work, k.slots, k.least), own_size = size_of(own_work, k.own_slots, k.least);

  // pieces before each group's and each sequence's, both in one scan
  const uint32_t n = (units + size - 1) / size, own_n = tid < batch ? max((own_units + own_size - 1) / own_size, 1u) : 0u;
  const u64 mine = (u64)(n * tiles) << 32 | own_n * k.own_tiles;
  u64 upto = wave_scan(mine);
  if (lane == 63) side3[wave] = upto;
  __syncthreads();
  u64 all = 0;
  for (uint32_t w = 0; w < threads / 64; ++w) {
    if (w < wave) upto += side3[w];
    all += side3[w];
  }
  upto -= mine;
  const uint32_t shared_items = (uint32_t)(all >> 32), own_items = (uint32_t)all;
  group_at[tid] = (uint32_t)(upto >> 32);
  own_at[tid] = (uint32_t)upto;
  if (tid == 0) {
    group_at[threads] = shared_items;
    own_at[threads] = own_items;
    k.counts[0] = shared_items;
    k.counts[1] = shared_items + own_items;
  }
  if (tid <= groups) k.ends[tid] = ends[tid];
  if (tid < groups) {
    k.common[tid] = common[tid];
    k.group_parts[tid] = make_uint2((uint32_t)(upto >> 32), n);
  }
  if (tid < batch) k.own_parts[tid] = make_uint2((uint32_t)upto, own_n);
  __syncthreads();
  // a thread to a piece: whose it is, by its place
  for (uint32_t i = tid; i < shared_items + own_items; i += threads) {
    const bool own = i >= shared_items;
    const uint32_t j = own ? i - shared_items : i;
    const uint32_t *at = own ? own_at : group_at;
    uint32_t low = 0, high = threads;   // at[low] <= j < at[high]
    while (high - low > 1) {
      const uint32_t mid = (low + high) / 2;
      if (at[mid] <= j) low = mid; else high = mid;
    }
    PrefixItem it;
    if (own) {
      const uint32_t part = (j - at[low]) / k.own_tiles;
      it.b = low;
      it.row0 = (j - at[low] - part * k.own_tiles) * k.own_tile;
      it.rows = per;
      it.first = first[low];
      it.ctx = lens[low] - it.first;
      it.tree = lives[low];
      it.lo = part * own_size;
      it.hi = min((it.ctx + 31) / 32 + (it.tree + 31) / 32, it.lo + own_size);
      it.turn = low + part;
      it.seq = seqs[low];
    } else {
      it.b = ends[low];
      it.rows = (ends[low + 1] - it.b) * per;
      const uint32_t t = (it.rows + k.tile - 1) / k.tile, part = (j - at[low]) / t;
      it.row0 = (j - at[low] - part * t) * k.tile;
      it.first = 0;
      it.ctx = common[low];
      it.tree = 0;
      it.lo = part * size;
      it.hi = min((it.ctx + 31) / 32, it.lo + size);
      it.turn = part;
      it.seq = seqs[it.b];
    }
    k.items[i] = it;
  }
}

// The same for any number of groups and sequences.
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
    uint32_t v = k.groups && g <= k.groups ? (uint32_t)max(0, min(k.starts[g], (int32_t)a.batch)) : 0u;
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

  u64 work = 0, own_work = 0, all = 0, own_all = 0;   // strips of all tiles of rows
  for (uint32_t g = tid; g < k.groups; g += kPlanThreads) {
    const uint32_t tiles = ((k.ends[g + 1] - k.ends[g]) * per + k.tile - 1) / k.tile;
    work += (u64)tiles * ((k.common[g] + 31) / 32);
  }
  for (uint32_t b = tid; b < a.batch; b += kPlanThreads) {
    const Seq q = sequence_of(a, b);
    own_work += (u64)k.own_tiles * ((q.len - k.first[b] + 31) / 32 + (q.live + 31) / 32);
  }
  group_scan(work, side64, all);
  group_scan(own_work, side64, own_all);
  const uint32_t size = size_of(all, k.slots, k.least), own_size = size_of(own_all, k.own_slots, k.least);

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
      it.turn = part;
      it.seq = tiles ? sequence_of(a, it.b).row : 0;
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
      it.seq = q.row;
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
      it.turn = b + part;
      k.items[slots + base + i] = it;
    }
    own += sum;
  }
  if (tid == 0) k.counts[1] = slots + own;
}

// A piece's numbers: the workgroup's, so scalars.
__device__ __forceinline__ PrefixItem item_of(const PrefixAttnArgs &k, uint32_t item) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(k.items + item);
  PrefixItem it;
  it.b = __builtin_amdgcn_readfirstlane(w[0]);
  it.row0 = __builtin_amdgcn_readfirstlane(w[1]);
  it.rows = __builtin_amdgcn_readfirstlane(w[2]);
  it.first = __builtin_amdgcn_readfirstlane(w[3]);
  it.ctx = __builtin_amdgcn_readfirstlane(w[4]);
  it.tree = __builtin_amdgcn_readfirstlane(w[5]);
  it.lo = __builtin_amdgcn_readfirstlane(w[6]);
  it.hi = __builtin_amdgcn_readfirstlane(w[7]);
  it.turn = __builtin_amdgcn_readfirstlane(w[8]);
  it.seq = __builtin_amdgcn_readfirstlane(w[9]);
  return it;
}

// Weights as the matrix unit takes them, eight of a lane: rounded to the values'
// type, and the rounded rest of each.
template <typename T> __device__ __forceinline__ uint4 rounded(const float (&p)[8]) {
  return make_uint4(pack2<T>(p[0], p[1]), pack2<T>(p[2], p[3]), pack2<T>(p[4], p[5]), pack2<T>(p[6], p[7]));
}
template <typename T> __device__ __forceinline__ uint4 rest_of(const float (&p)[8], uint4 r) {
  const auto two = [](float a, float b, uint32_t w) { return pack2<T>(a - half_of<T>(w, 0), b - half_of<T>(w, 1)); };
  return make_uint4(two(p[0], p[1], r.x), two(p[2], p[3], r.y), two(p[4], p[5], r.z), two(p[6], p[7], r.w));
}

// (x - top) unit for scores of any size: their halves differ by a finite number.
__device__ __forceinline__ float less_of(float x, float top, float unit) {
  return fmaf(x, 0.5f, -0.5f * top) * (2.f * unit);
}
// Where a cached token's row lies, in 16-byte units.
__device__ __forceinline__ uint32_t cached_row(const PrefixAttnArgs &k, const int32_t *table, uint32_t key) {
  const uint32_t entry = k.page.quot(key), page = min((uint32_t)max(table[entry], 0), k.a.n_pages - 1);
  return page * (uint32_t)(k.a.cache_page / 8) + (key - entry * k.page.d) * (uint32_t)(k.a.cache_token / 8);
}
// Adds those values that are no finite numbers, N runs of C; a run is live(n) or
// not there. Rarely is there one.
template <typename T, int N, int C, typename L>
__device__ __forceinline__ void add_nonfinite(const T *row, int stride, L live, float (&sum)[N][C]) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  constexpr uint32_t E = Half<T>::kExp;
  uint32_t w[N][C / 2];
  u16x2 top = {0, 0};   // greatest exponents
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if constexpr (C == 8) {
      const uint4 v = live(n) ? *reinterpret_cast<const uint4 *>(row + n * stride) : make_uint4(0, 0, 0, 0);
      w[n][0] = v.x, w[n][1] = v.y, w[n][2] = v.z, w[n][3] = v.w;
    } else {
      const uint2 v = live(n) ? *reinterpret_cast<const uint2 *>(row + n * stride) : make_uint2(0, 0);
      w[n][0] = v.x, w[n][1] = v.y;
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[n][i] & (E | E << 16)));
  if (top.x != E && top.y != E) return;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float x = half_of<T>(w[n][i / 2], i & 1);
      if (!__builtin_isfinite(x)) sum[n][i] += x;
    }
}

// ---- a piece

// U: 16-row units of the tile. EXACT: head_dim is DP. OWN: the sequence's own
// tokens and its tree; else shared ones.
template <typename T, int DP, int U, bool EXACT, bool OWN>
__device__ __forceinline__ void piece(const PrefixAttnArgs &k, const PrefixItem &it, uint32_t h, uint64_t at, float *joint) {
  constexpr int KS = DP / 32;                   // k steps of Q K^T
  constexpr int C = DP >= 128 ? 8 : DP / 16;    // consecutive values a lane transposes
  constexpr int NH = DP / (16 * C);             // groups of 16 C values
  constexpr int NREG = U * NH * C * 4;          // accumulators a lane holds
  const enc_tree_attention_args &a = k.a;
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l16 = lane & 15, g4 = lane >> 4;
  const uint32_t D = a.head_dim;
  const uint32_t b0 = it.b, first = OWN ? it.first : 0, ctx = it.ctx;
  const int32_t *table = a.d_table + (uint64_t)it.seq * a.max_pages;
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

  // m: half the maximum of q.k, before the scale. Halves of two finite scores
  // differ by a finite number, so scale 0 and the least scales are like others.
  f32x4 o[U][NH][C];
  float m[U], l[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = 0.5f * kLowest;
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
  uint32_t ko[2], vo[8];   // of the keys that this lane loads, got from the lanes that know them
  auto offsets_of = [&](uint32_t strip, int32_t e) {
    uint32_t k_at, v_at;
    if (!OWN || strip < strips_ctx) {
      const uint32_t key = first + min(strip * 32 + (lane & 31), ctx - 1), page = min((uint32_t)max(e, 0), a.n_pages - 1);
      k_at = v_at = page * page_units + (key - k.page.quot(key) * k.page.d) * token_units;
    } else {
      const uint32_t key = min((strip - strips_ctx) * 32 + (lane & 31), it.tree - 1);
      k_at = key * (uint32_t)(a.k_new_node / 8);
      v_at = key * (uint32_t)(a.v_new_node / 8);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) ko[t] = (uint32_t)__shfl((int)k_at, 16 * t + l16);
#pragma unroll
    for (int j = 0; j < 8; ++j) vo[j] = (uint32_t)__shfl((int)v_at, 16 * (j >> 2) + 4 * g4 + (j & 3));
  };
  auto load_k = [&](uint32_t strip) {
    const uint4 *base = !OWN || strip < strips_ctx ? kc : reinterpret_cast<const uint4 *>(kn);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint4 *p = base + ko[t];
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
  auto load_v = [&](uint32_t strip) {
    const uint4 *base = !OWN || strip < strips_ctx ? vc : reinterpret_cast<const uint4 *>(vn);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 *p = base + vo[j];
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
  const float c2 = 2.f * k.unit, slack = k.half_slack;
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
    __builtin_amdgcn_sched_barrier(0);   // the next strip's K into the same registers
    after_k();
    __builtin_amdgcn_sched_barrier(0);

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

    uint4 pf[U], pl[U];
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
      top = 0.5f * rows_max(top);
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
        p[u][j] = __builtin_amdgcn_exp2f(fmaf(fmaf(p[u][j], 0.5f, -m[u]), c2, Half<T>::kLift2));
        if constexpr (SPECIAL)   // -infinity times a scale of 0 is no number
          if (!(seen[u] >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = 0.f;
      }
      l[u] += ((p[u][0] + p[u][1]) + (p[u][2] + p[u][3])) + ((p[u][4] + p[u][5]) + (p[u][6] + p[u][7]));
      pf[u] = rounded<T>(p[u]);
      pl[u] = rest_of<T>(p[u], pf[u]);
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
          o[u][n][f] = Half<T>::mfma(vf, pl[u], o[u][n][f]);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
    after_v();
    __builtin_amdgcn_sched_barrier(0);
  };

  // Whole strips of cached keys but the wave's last: every one loads the next
  // without asking whether there is one (a branch around loads makes the waits
  // behind it wait for all of them). The last whole strip, the one that is not
  // full and the tree's follow, one load at a time.
  const uint32_t whole = min(hi, ctx / 32);
  uint32_t strip = lo + wave;
  if (strip < hi) {
    offsets_of(strip, entry_of(strip));
    // in the loop's order, or its waits allow for both
    load_k(strip);
    __builtin_amdgcn_sched_barrier(0);
    int32_t entry = entry_of(min(strip + kWays, hi - 1));
    __builtin_amdgcn_sched_barrier(0);
    load_v(strip);
    __builtin_amdgcn_sched_barrier(0);
    while (strip + kWays < whole) {
      const uint32_t next = strip + kWays;
      offsets_of(next, entry);
      compute(
          std::false_type{}, strip,
          [&] {
            load_k(next);
            entry = entry_of(min(next + kWays, hi - 1));
          },
          [&] { load_v(next); });
      strip = next;
    }
    while (true) {
      compute(std::true_type{}, strip, [] {}, [] {});
      strip += kWays;
      if (strip >= hi) break;
      offsets_of(strip, entry_of(strip));
      load_k(strip);
      load_v(strip);
    }
  }
  // The rest of a weight may be 0 or below, and so may come no number, or the
  // wrong infinity, of an infinite cached value. Every row sees that: where no row
  // is finite, though the weights of some are, the values at fault are looked for
  // and their sum is the result (16 sequences over 131072 tokens then take 2.2 ms).
  bool lost = true, weighed = false;
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
    weighed = weighed || __builtin_isfinite(rows_sum(l[u]));
  }
  if (__all(lost) && __any(weighed)) {
    float sum[NH][4][1][C] = {};
    for (strip = lo + wave; strip < min(hi, strips_ctx); strip += kWays) {
      const uint32_t at = cached_row(k, table, first + min(strip * 32 + (lane & 31), ctx - 1));
#pragma unroll 4
      for (int key = 0; key < 32; ++key) {   // (the last one more than once)
        const T *row = reinterpret_cast<const T *>(vc + (uint32_t)__shfl((int)at, key));
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t d = (n * 16 + 4 * g4 + i) * C;
            add_nonfinite(row + d, 0, [&](int) { return EXACT || d < D; }, sum[n][i]);
          }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float none = 0.f * rows_sum(l[u]);   // a row of its own fault stays no number
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int f = 0; f < C; ++f)
            if (sum[n][i][0][f] != 0.f) o[u][n][f][i] = sum[n][i][0][f] + none;
    }
  }
  // Infinities and NaN of the tree went in as zeros, since 0 times them would
  // reach rows that do not see them: add them to the rows that do.
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
    if (g4 == 0) *reinterpret_cast<float2 *>(k.part_ml + 2 * row) = make_float2(2.f * m[u], l[u]);
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

// The pieces from item0 on. UP, US: units of a tile of shared (0: another kernel
// takes those) and of own tokens' rows.
template <typename T, int DP, int UP, int US, bool EXACT>
__global__ __launch_bounds__(256, (DP == 256 ? 1 : UP + US == 1 ? 3 : 2)) void k_pieces(PrefixAttnArgs k) {
  constexpr int U = UP > US ? UP : US;
  __shared__ float joint[2 * (U * DP / 4 + 2 * U) * 64];
  const uint32_t shared = __builtin_amdgcn_readfirstlane(k.counts[0]), heads = k.a.kv_heads;
  const uint32_t at = blockIdx.x / heads, item = UP ? at : at + shared;
  const PrefixItem it = item_of(k, item);   // on its way with the count
  if (item >= __builtin_amdgcn_readfirstlane(k.counts[1])) return;
  // Neighbouring workgroups differ in their head; with 8 heads the tiles of a
  // range meet on one die and in its L2.
  const uint32_t h = (blockIdx.x - at * heads + it.turn) % heads;
  if constexpr (UP)
    if (item < shared) {
      piece<T, DP, UP, EXACT, false>(k, it, h, ((uint64_t)item * heads + h) * (16 * UP), joint);
      return;
    }
  piece<T, DP, US, EXACT, true>(k, it, h, k.own_rows + ((uint64_t)(item - shared) * heads + h) * (16 * US), joint);
}

// ---- pieces of shared tokens with many rows: K and V through LDS
//
// Eight waves: four tiles of U units of rows, two at different keys. A stage of
// 64 keys is brought in by all of them and read by each, 32 keys of it, so that
// a range's sums are joined over two waves and its rows written once: with eight
// tiles of rows on the same keys there would be twice the partial sums, which
// cost as much HBM traffic as the keys themselves at 256 rows and 8192 tokens.
// Direct loads into fragments, as in `piece`, take a cache line for every 16
// bytes of K: 64 rows and more wait for that. Heads up to 128 values: three
// stages lie in LDS (the one computed, the next, whose first K fragments are read
// early, and the one a slower wave may still be in), a fourth is on its way into
// registers. Above: two, for want of registers and LDS. Banks: a wave reads one
// 16-byte chunk of 16 rows of K at a time, so chunk c of row r lies at
// c ^ k_turn(r); of V it reads 32 bytes of 8 rows, so rows lie 32 bytes further
// apart than they are long. V^T fragments come from ds_read_b64_tr.
template <int NCH> __device__ __forceinline__ constexpr uint32_t k_turn(uint32_t r) {
  return NCH == 8 ? r >> 1 & 7 : r & 15;   // 16 rows (two to 256 bytes, for 8 chunks) on 16 places
}

constexpr uint32_t kStage = 64;      // keys of a stage
constexpr float kFar = 65536.f;      // see below

template <typename T, int DP, int U>
__global__ __launch_bounds__(512, 2) void k_shared(PrefixAttnArgs k) {
  constexpr int KS = DP / 32, NF = DP / 16, NCH = DP / 8;
  constexpr bool PIPE = DP <= 128;                 // registers for a strip's K and V fragments at once
  constexpr uint32_t NB = PIPE ? 3 : 2;            // stages in LDS
  constexpr int NT = 512, NR = kStage * NCH / NT;  // chunks of K (and of V) a thread brings in
  constexpr int PITCH = NCH + 2;                   // 16-byte chunks from row to row of V
  constexpr uint32_t kRows = 64 * U;               // of the tile
  const enc_tree_attention_args &a = k.a;
  __shared__ __align__(16) uint4 room[NB * kStage * (NCH + PITCH)];
  uint4 *const ks = room, *const vs = room + NB * kStage * NCH;

  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t l16 = lane & 15, g4 = lane >> 4, half = wave >> 2;   // the strip of a stage that is this wave's
  const uint32_t D = a.head_dim, heads = a.kv_heads, item = blockIdx.x / heads;
  const PrefixItem it = item_of(k, item);   // on its way with the count
  if (item >= __builtin_amdgcn_readfirstlane(k.counts[0])) return;
  const uint32_t h = (blockIdx.x - item * heads + it.turn) % heads, ctx = it.ctx;
  const uint32_t lo = it.lo / 2, hi = (it.hi + 1) / 2;   // stages
  const int32_t *table = a.d_table + (uint64_t)it.seq * a.max_pages;

  const uint32_t first_row = it.row0 + (wave & 3) * (16 * U);
  const bool busy = first_row < it.rows;   // this wave has rows
  uint4 qf[U][KS];
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;   // -scale (-q).k
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = first_row + 16 * u + l16, rr = min(r, it.rows - 1);
    const uint32_t turn = k.group.quot(rr), member = k.nodes.quot(turn), node = turn - member * a.nodes;
    const uint32_t head = h * k.group.d + (rr - turn * k.group.d);
    const T *p = static_cast<const T *>(a.d_q) + (it.b + member) * a.q_batch + node * a.q_node + head * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t d = 32 * s + 8 * g4;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < it.rows && d < D) v = *reinterpret_cast<const uint4 *>(p + d);
      qf[u][s] = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
    }
  }
  // A key's weight is 2^(p c2 - mc), p = q.k: one fma, exact until it is rounded,
  // so that mc, the row's maximum mr times c2 (less the lift), may be rounded as
  // it likes. From kFar on the rounding of mc alone is no longer small beside 1:
  // there it is 2^((p - mr) c2), whose difference is exact where it is small.
  const float c2 = k.unit, slack = k.slack;
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
  constexpr uint32_t kRowStep = NT / NCH;
  const bool chunk_live = ch * 8 < D;
  // One or two stages are on their way into registers while another waits in LDS. Loads
  // are never behind a branch (one would make the waits behind it wait for all):
  // stages past the last stand for the last, keys past the end for the last one,
  // and what is no key's becomes 0 when it is placed.
  const uint4 *kc = static_cast<const uint4 *>(a.d_k_cache) + h * (a.cache_head / 8) + (chunk_live ? ch : 0);
  const uint4 *vc = static_cast<const uint4 *>(a.d_v_cache) + h * (a.cache_head / 8) + (chunk_live ? ch : 0);
  const uint32_t page_units = (uint32_t)(a.cache_page / 8), token_units = (uint32_t)(a.cache_token / 8);
  constexpr uint32_t kAhead = 2;      // stages on their way: registers
  uint4 kr[kAhead][NR], vr[kAhead][NR];
  const uint32_t whole_end = min(hi, ctx / kStage);   // stages from here on are not full
  const bool part = D != DP;
  auto entry_of = [&](uint32_t st) { return table[k.page.quot(min(min(st, hi - 1) * kStage + lane, ctx - 1))]; };
  auto fetch = [&](auto slot_, uint32_t st, int32_t entry) __attribute__((always_inline)) {   // entry: for key lane
    constexpr int S = decltype(slot_)::value;
    const uint32_t key = min(min(st, hi - 1) * kStage + lane, ctx - 1), page = min((uint32_t)max(entry, 0), a.n_pages - 1);
    const uint32_t at = page * page_units + (key - k.page.quot(key) * k.page.d) * token_units;
    uint32_t off[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) off[i] = (uint32_t)__shfl((int)at, r0 + i * kRowStep);
#pragma unroll
    for (int i = 0; i < NR; ++i) kr[S][i] = kc[off[i]];
#pragma unroll
    for (int i = 0; i < NR; ++i) vr[S][i] = vc[off[i]];
    __builtin_amdgcn_sched_barrier(0);
  };
  auto place = [&](auto slot_, uint32_t st, uint32_t buf) __attribute__((always_inline)) {
    constexpr int S = decltype(slot_)::value;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint32_t r = r0 + i * kRowStep;
      uint4 kv = kr[S][i], vv = vr[S][i];
      if (part || st >= whole_end) {   // a branch, not selects on every stage's way
        asm volatile("");
        if (!chunk_live || st * kStage + r >= ctx) kv = vv = make_uint4(0, 0, 0, 0);
      }
      ks[(buf * kStage + r) * NCH + (ch ^ k_turn<NCH>(r))] = kv;
      vs[(buf * kStage + r) * PITCH + ch] = vv;
    }
  };

  // New maxima where a strip exceeds the old ones, and what is summed so far
  // brought to them; other rows stay as they are, to the bit.
  auto grow = [&](const float (&top)[U]) __attribute__((always_inline)) {
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

  float p[U][8], top[U];
  uint4 kf[2][KS];
  auto read_k = [&](uint32_t buf) {
    const uint4 *row = ks + (buf * kStage + half * 32 + l16) * NCH;
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
  auto values_at = [&](uint32_t buf) {
    return reinterpret_cast<const char *>(vs + (buf * kStage + half * 32 + 4 * g4 + (l16 >> 2)) * PITCH) + (l16 & 3) * 8;
  };
  // The weights of a strip whose maxima are known, packed, and their rests; l grows
  // by them. With `masked` only the keys of `bits` weigh anything. `between`: what
  // runs beside the exponentials.
  auto weigh = [&](auto masked_, uint32_t bits, uint4 (&pf)[U], uint4 (&pl)[U], auto between) __attribute__((always_inline)) {
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
    between();
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[u][j] = __builtin_amdgcn_exp2f(fmaf(p[u][j], c2, -off[u]));
        if constexpr (decltype(masked_)::value)   // -infinity times a scale of 0 is no number
          if (!(bits >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = 0.f;
      }
      l[u] += ((p[u][0] + p[u][1]) + (p[u][2] + p[u][3])) + ((p[u][4] + p[u][5]) + (p[u][6] + p[u][7]));
      pf[u] = rounded<T>(p[u]);
      pl[u] = rest_of<T>(p[u], pf[u]);
    }
  };

  // ---- a strip by itself: the last ones, and heads above 128 values
  auto compute = [&](uint32_t st, uint32_t buf) __attribute__((always_inline)) {
    const uint32_t from = st * kStage + half * 32;
    const uint32_t bits = ctx >= from + 32 ? 0xFFFFFFFFu : ctx <= from ? 0u : (1u << (ctx - from)) - 1u;
    if constexpr (PIPE) {
      read_k(buf);
      scores(p);
    } else {   // half of K at a time: registers
      const uint4 *row = ks + (buf * kStage + half * 32 + l16) * NCH;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < KS; ++e) {
          const uint4 f = row[16 * t * NCH + ((4 * e + g4) ^ k_turn<NCH>(l16))];
#pragma unroll
          for (int u = 0; u < U; ++u) s[u] = Half<T>::mfma(f, qf[u][e], s[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[u][4 * t + e] = s[u][e];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(bits >> (16 * (j >> 2) + 4 * g4 + (j & 3)) & 1u)) p[u][j] = -__builtin_inff();
    maxima();
    uint4 pf[U], pl[U];
    weigh(std::true_type{}, bits, pf, pl, [] {});
    const char *vb = values_at(buf);
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint2 v0 = read_transposed(vb + 32 * f), v1 = read_transposed(vb + 16 * PITCH * 16 + 32 * f);
      const uint4 vf = make_uint4(v0.x, v0.y, v1.x, v1.y);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        o[u][f] = Half<T>::mfma(vf, pf[u], o[u][f]);
        o[u][f] = Half<T>::mfma(vf, pl[u], o[u][f]);
      }
    }
  };

  // ---- whole strips, two in flight: while the exponentials of one are taken,
  // the products of the next with K run, and while its products with V run, the
  // next's maxima are taken
  auto step = [&](uint32_t buf, uint32_t k_buf) __attribute__((always_inline)) {
    if constexpr (PIPE) {
      read_k(k_buf);
      float x[U][8];
      uint4 pf[U], pl[U];
      weigh(std::false_type{}, 0u, pf, pl, [&] {
        __builtin_amdgcn_sched_barrier(0);
        scores(x);
      });
#pragma unroll
      for (int i = 0; i < 2 * KS * U; ++i) {   // a product, then a few of the others, in turn
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) p[u][j] = x[u][j];
      const char *vb = values_at(buf);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint2 v0 = read_transposed(vb + 32 * f), v1 = read_transposed(vb + 16 * PITCH * 16 + 32 * f);
        const uint4 vf = make_uint4(v0.x, v0.y, v1.x, v1.y);
#pragma unroll
        for (int u = 0; u < U; ++u) o[u][f] = Half<T>::mfma(vf, pf[u], o[u][f]);
#pragma unroll
        for (int u = 0; u < U; ++u) o[u][f] = Half<T>::mfma(vf, pl[u], o[u][f]);
      }
      maxima();
#pragma unroll
      for (int i = 0; i < 2 * NF * U; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // A stage's turn. With PIPE the next one is placed ahead of it (its first K is
  // read before the other's end), else the stage itself.
  uint32_t st = lo, buf = 0;
  int32_t entry;   // of the stage that is fetched next
  auto turn_of = [&](auto slot_) __attribute__((always_inline)) {
    constexpr int S = decltype(slot_)::value;
    const uint32_t next = buf + 1 == NB ? 0 : buf + 1;
    if constexpr (PIPE) {
      place(std::integral_constant<int, S>{}, st + 1, next);
      fetch(std::integral_constant<int, S>{}, st + 1 + kAhead, entry);
      entry = entry_of(st + 2 + kAhead);
      __syncthreads();
      if (busy) step(buf, st + 1 < whole_end ? next : buf);   // else: products that nobody asks for
    } else {
      place(std::integral_constant<int, S>{}, st, buf);
      fetch(std::integral_constant<int, S>{}, st + kAhead, entry);
      entry = entry_of(st + 1 + kAhead);
      __syncthreads();
      if (busy) compute(st, buf);
    }
    buf = next;
    ++st;
  };
  constexpr int kOther = kAhead - 1;
  const int32_t e0 = entry_of(lo), e1 = entry_of(lo + 1), e2 = entry_of(lo + 2);
  __builtin_amdgcn_sched_barrier(0);
  fetch(std::integral_constant<int, 0>{}, lo, e0);
  if constexpr (kAhead == 2) fetch(std::integral_constant<int, 1>{}, lo + 1, e1);
  if constexpr (PIPE) {
    place(std::integral_constant<int, 0>{}, lo, 0);
    fetch(std::integral_constant<int, 0>{}, lo + kAhead, kAhead == 2 ? e2 : e1);
    entry = entry_of(lo + 1 + kAhead);
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    if (st < whole_end) {
      if (busy) {
        read_k(0);
        scores(p);
        maxima();
      }
      while (true) {
        turn_of(std::integral_constant<int, kOther>{});
        if (st >= whole_end) break;
        if constexpr (kAhead == 2) {
          turn_of(std::integral_constant<int, 0>{});
          if (st >= whole_end) break;
        }
      }
    }
    if (st < hi) {   // one that is not full
      __syncthreads();
      if (busy) compute(st, buf);
    }
  } else {
    entry = kAhead == 2 ? e2 : e1;
    while (true) {
      turn_of(std::integral_constant<int, 0>{});
      if (st >= hi) break;
      if constexpr (kAhead == 2) {
        turn_of(std::integral_constant<int, 1>{});
        if (st >= hi) break;
      }
    }
  }

  // As in `piece`: infinite values, of the keys that were this wave's.
  bool lost = busy, weighed = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float zero = 0.f;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) zero = fmaf(o[u][f][e], 0.f, zero);
    lost = lost && rows_sum(zero) != 0.f;
    weighed = weighed || __builtin_isfinite(rows_sum(l[u]));
  }
  if (__all(lost) && __any(weighed)) {
    const uint4 *values = static_cast<const uint4 *>(a.d_v_cache) + h * (a.cache_head / 8);
    float sum[NF / 4][4][4] = {};
    for (st = lo; st < hi && st * kStage + half * 32 < ctx; ++st) {
      const uint32_t at = cached_row(k, table, min(st * kStage + half * 32 + (lane & 31), ctx - 1));
#pragma unroll 2
      for (int key = 0; key < 32; ++key) {
        const T *row = reinterpret_cast<const T *>(values + (uint32_t)__shfl((int)at, key));
#pragma unroll
        for (int n = 0; n < NF / 4; ++n)
          add_nonfinite(row + 64 * n + 4 * g4, 16, [&](int f) { return 64 * n + 16 * f + 4 * g4 < D; }, sum[n]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float none = 0.f * rows_sum(l[u]);
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (sum[f / 4][f % 4][e] != 0.f) o[u][f][e] = sum[f / 4][f % 4][e] + none;
    }
  }

  // ---- join the two waves of a tile, write
  constexpr uint32_t kLane = U * (4 * NF + 2);   // numbers of a lane
  static_assert(kLane * 64 * 4 * 4 <= sizeof(room), "the sums of four waves fit the stages' room");
  float *const mine = reinterpret_cast<float *>(room) + (wave & 3) * kLane * 64 + lane;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // sums of weights 2^((p - mr) c2 + lift), whichever way they were taken
    const float fix = beyond(u) ? 1.f : __builtin_amdgcn_exp2f(fmaf(-mr[u], c2, mc[u]) + Half<T>::kLift2);
    l[u] = rows_sum(l[u]) * fix;
    mr[u] = fmaxf(mr[u], kLowest);
#pragma unroll
    for (int f = 0; f < NF; ++f) o[u][f] *= fix;
  }
  __syncthreads();
  if (half == 1) {
    uint32_t i = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mine[64 * i++] = mr[u];
      mine[64 * i++] = l[u];
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) mine[64 * i++] = o[u][f][e];
    }
  }
  __syncthreads();
  if (half == 1 || !busy) return;
  uint32_t i = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float m2 = mine[64 * i++], l2 = mine[64 * i++];
    const float up = fmaxf(mr[u], m2);
    const float w1 = __builtin_amdgcn_exp2f(less_of(mr[u], up, c2)), w2 = __builtin_amdgcn_exp2f(less_of(m2, up, c2));
    l[u] = l[u] * w1 + l2 * w2;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[u][f][e] = o[u][f][e] * w1 + mine[64 * i++] * w2;
    if (first_row + 16 * u + l16 >= it.rows) continue;
    const uint64_t row = ((uint64_t)item * heads + h) * kRows + (wave & 3) * (16 * U) + 16 * u + l16;
    if (g4 == 0) *reinterpret_cast<float2 *>(k.part_ml + 2 * row) = make_float2(up, l[u]);
    float *dst = k.part + row * D;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const uint32_t d = 16 * f + 4 * g4;
      if (d < D) *reinterpret_cast<f32x4 *>(dst + d) = o[u][f];
    }
  }
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
    const float w = __builtin_amdgcn_exp2f(less_of(part.x, m, k.unit));
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
void launch_pieces(const PrefixAttnArgs &k, uint32_t items, hipStream_t s) {
  const dim3 grid(items * k.a.kv_heads), block(256);
  if (k.a.head_dim == DP)
    hipLaunchKernelGGL((k_pieces<T, DP, UP, US, true>), grid, block, 0, s, k);
  else
    hipLaunchKernelGGL((k_pieces<T, DP, UP, US, false>), grid, block, 0, s, k);
}

template <typename T, int DP>
void launch_dim(const PrefixAttnArgs &k, const PrefixAttnPlan &p, hipStream_t s) {
  constexpr int US = DP <= 128 ? 2 : 1;   // units of many own rows
  if (k.groups && p.tile == 16) {
    launch_pieces<T, DP, 1, 1>(k, p.items, s);
    return;
  }
  if (k.groups) {   // (else nothing is shared)
    const dim3 grid(p.most_shared * k.a.kv_heads), block(512);
    if (p.tile == 64)
      hipLaunchKernelGGL((k_shared<T, DP, 1>), grid, block, 0, s, k);
    else if constexpr (DP <= 128)
      hipLaunchKernelGGL((k_shared<T, DP, 2>), grid, block, 0, s, k);
  }
  if (p.own_tile == 16)
    launch_pieces<T, DP, 0, 1>(k, p.most_own, s);
  else if constexpr (US > 1)
    launch_pieces<T, DP, 0, US>(k, p.most_own, s);
}

template <typename T>
void launch_type(const PrefixAttnArgs &k, const PrefixAttnPlan &p, hipStream_t s) {
  const uint32_t D = k.a.head_dim, rows = k.a.batch * k.a.nodes * k.a.q_heads;
  if (k.a.batch <= kPlanThreads && k.groups < kPlanThreads)
    hipLaunchKernelGGL(k_prefix_plan_small, dim3(1), dim3((std::max({k.a.batch, k.groups + 1, 256u}) + 63) / 64 * 64), 0, s, k);
  else
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

// ---- how many leading tokens the sequences of a group have in common
__global__ __launch_bounds__(kPlanThreads) void k_cache_shared(enc_cache c, const int32_t *seqs, uint32_t batch,
                                                               const int32_t *starts, int32_t *shared) {
  __shared__ uint32_t bottom, least, differs;
  const uint32_t g = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) bottom = 0, least = differs = ~0u;
  __syncthreads();
  const auto clamped = [&](uint32_t i) { return (uint32_t)max(0, min(starts[i], (int32_t)batch)); };
  uint32_t from = 0;
  for (uint32_t i = tid; i <= g; i += kPlanThreads) from = max(from, clamped(i));
  for (uint32_t o = 32; o; o >>= 1) from = max(from, (uint32_t)__shfl_xor((int)from, o));
  if ((tid & 63) == 0) atomicMax(&bottom, from);   // (64 lanes with values of their own would go one by one)
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
  for (uint32_t o = 32; o; o >>= 1) len = min(len, (uint32_t)__shfl_xor((int)len, o));
  if ((tid & 63) == 0) atomicMin(&least, len);
  __syncthreads();
  len = least;
  const uint32_t pages = (len + c.page_size - 1) / c.page_size;
  // A wave to four sequences, 256 entries of each at a time, all on their way at
  // once, up to the first that differs from the group's first sequence's. (len is
  // not 0 below: every sequence is one of the table.)
  const int32_t *row0 = c.d_table + (uint64_t)(uint32_t)seqs[from] * c.max_pages;
  const uint32_t lane = tid & 63;
  for (uint32_t b = from + (tid >> 6) * 4; b < to; b += kPlanThreads / 64 * 4) {
    const int32_t *row[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) row[i] = c.d_table + (uint64_t)(uint32_t)seqs[min(b + i, to - 1)] * c.max_pages;
    const uint32_t end = min(pages, differs);   // (others may lower it meanwhile)
    for (uint32_t p0 = 0; p0 < end; p0 += 256) {
      bool odd[4] = {false, false, false, false};
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t p = min(p0 + 64 * e + lane, pages - 1);
        const int32_t want = row0[p];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const int32_t own = row[i][p];
          odd[e] |= own < 0 || own != want;
        }
      }
      uint32_t at = ~0u;
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        const uint64_t hit = __ballot(odd[e]);
        if (hit) at = p0 + 64 * e + __builtin_ctzll(hit);
      }
      if (at != ~0u) {
        if (lane == 0) atomicMin(&differs, min(at, pages));
        break;
      }
    }
  }
  __syncthreads();
  if (tid == 0) shared[g] = (int32_t)min((uint64_t)min(differs, pages) * c.page_size, (uint64_t)len);
}

}  // namespace

namespace {

// Average rows of a group from which tiles are of 64 and of 128 rows, and rows of
// a sequence from which its own are of 32.
//
// A tile of shared tokens that has rows to spare, or two tiles that each read the
// keys, cost more by the token; a call of less than some ten microseconds more of
// them starts later with the larger one (its first stage, the exchange between its
// waves, what it writes). Whole calls in us, 8 KV heads of 128, for 1021 / 8192 /
// 131072 shared tokens in tiles of 16, 64 and 128:
//     32 rows: 16.5 / 27.6 / 140, 23.1 / 32.1 / 123, 25.1 / 34.9 / 131;
//     64 rows: 18.5 / 30.4 / 218, 24.8 / 34.7 / 124, 26.4 / 36.6 / 134;
//    128 rows: 23.7 / 38.1 / 369, 26.1 / 37.4 / 181, 29.4 / 41.1 / 160;
//    256 rows: 27.9 / 59.1 / 644, 31.0 / 45.8 / 309, 33.9 / 46.7 / 258;
//   1024 rows: 60.6 / 175 / -, 52.9 / 110 / -, 55.7 / 99 / -.
// So the rule costs up to a third where 33 to 256 rows share some 1000 tokens, 10 to
// 14% where 33 to 64 share 8192, and up to 2% otherwise. What a sequence's
// table can hold stands for its length, which the host does not know: in a table
// far wider than the histories a call takes the figures of the longer ones' tiles.
//
// Of own tokens, in tiles of 16 and of 32 rows: 32 rows of a sequence 32.5 and 35.7
// us (16 sequences of 8 nodes, 1000 own tokens, heads of 128), 25.6 and 25.7 with
// heads of 64 (40 sequences, 300 tokens); 64 rows 42.3 and 40.4, heads of 64 35.7
// and 37.2; 256 rows 91.6 and 77.6.
struct TileRule {
  bool large;   // heads above 128 values: no tiles of 128 rows, nor of 32 own ones
  uint64_t from64, from128, own32;
};
TileRule tile_rule(const enc_tree_attention_args &a) {
  const uint64_t room = (uint64_t)a.max_pages * a.page_size;
  return {a.head_dim > 128, room > 32768 ? 17u : 33u, room > 16384 ? 65u : 129u, a.head_dim > 64 ? 33u : 17u};
}

// The plan for given tiles: pieces of `slots` equal shares of the work, and one
// more, a short one, for every tile.
//
// Resident workgroups: one of eight waves to a compute unit, or two or three of
// four. 64 sequences over 8192 shared tokens take 66.7 us; with twice as many
// shares of the shared tokens 78.2, with three quarters 70.2; with half or twice
// as many shares of the own ones 66.7 and 65.7.
PrefixAttnPlan plan_of(const enc_tree_attention_args &a, uint32_t groups, uint32_t tile, uint32_t own_tile,
                       uint64_t tiles, uint64_t own_tiles_of_all) {
  PrefixAttnPlan p;
  p.tile = tile;
  p.own_tile = own_tile;
  p.own_tiles = (a.nodes * (a.q_heads / a.kv_heads) + own_tile - 1) / own_tile;
  p.slots = std::max((tile == 16 ? 512 : 256) / a.kv_heads, 1u);
  p.own_slots = std::max(768 / a.kv_heads, 1u);
  p.least = kWays;
  p.most_shared = groups ? (uint32_t)(p.slots + tiles) : 0;
  p.most_own = (uint32_t)(p.own_slots + own_tiles_of_all);
  p.items = p.most_shared + p.most_own;
  const uint64_t n = (uint64_t)p.most_shared * a.kv_heads * p.tile + (uint64_t)p.most_own * a.kv_heads * p.own_tile;
  p.part_bytes = align_up(4 * n * a.head_dim, 256);
  p.ml_bytes = align_up(8 * n, 256);
  p.item_bytes = align_up(sizeof(PrefixItem) * (uint64_t)p.items, 256);
  p.batch_bytes = align_up(4ull * a.batch, 256);
  p.group_bytes = align_up(4ull * (groups + 1), 256);
  return p;
}

}  // namespace

PrefixAttnPlan plan_prefix_attention(const enc_tree_attention_args &a, uint32_t groups) {
  const TileRule rule = tile_rule(a);
  const uint32_t per = a.nodes * (a.q_heads / a.kv_heads);
  const uint64_t rows = (uint64_t)a.batch * per, mean = rows / std::max(groups, 1u);
  const uint32_t tile = !groups ? 16 : mean >= rule.from128 && !rule.large ? 128 : mean >= rule.from64 ? 64 : 16;
  // (with tiles of 16 one kernel takes both)
  const uint32_t own_tile = per >= rule.own32 && !rule.large && (!groups || tile > 16) ? 32 : 16;
  return plan_of(a, groups, tile, own_tile, std::min<uint64_t>(rows / tile + groups, rows),
                 (uint64_t)a.batch * ((per + own_tile - 1) / own_tile));
}

// Enough for every call with no more sequences, nodes, groups or room in the
// table: fewer groups have larger tiles, so the most over the tiles that such calls
// can choose, each with as many of them as there can be.
uint64_t prefix_attention_bytes(const enc_tree_attention_args &a, uint32_t groups) {
  const TileRule rule = tile_rule(a);
  const uint32_t per = a.nodes * (a.q_heads / a.kv_heads);
  const uint64_t rows = (uint64_t)a.batch * per;
  uint64_t most = 0;
  const auto consider = [&](uint32_t any, uint32_t tile, uint32_t own_tile, uint64_t tiles, uint64_t own) {
    most = std::max(most, plan_of(a, any, tile, own_tile, tiles, own).total());
  };
  for (uint32_t own_tile = 16; own_tile <= (per >= rule.own32 && !rule.large ? 32u : 16u); own_tile += 16) {
    const uint64_t own = (uint64_t)a.batch * ((per + own_tile - 1) / own_tile);
    consider(0, 16, own_tile, 0, own);
    if (!groups) continue;
    if (own_tile == 16) {
      const uint64_t few = std::min<uint64_t>(rows, 33ull * groups);   // at most 32 rows a group, on average
      consider(groups, 16, 16, std::min<uint64_t>(few / 16 + groups, few), std::min(own, few));
    }
    if (rows >= rule.from64)
      consider(groups, 64, own_tile, rows / 64 + std::min<uint64_t>(groups, rows / rule.from64), own);
    if (rows >= rule.from128 && !rule.large)
      consider(groups, 128, own_tile, rows / 128 + std::min<uint64_t>(groups, rows / rule.from128), own);
  }
  return most;
}

hipError_t launch_prefix_attention(PrefixAttnArgs k, const PrefixAttnPlan &p, hipStream_t s) {
  k.unit = std::min(std::fabs(k.a.scale) * kLog2e, -kLowest / 2);   // (twice that is used)
  k.slack = std::min(kSlack2 / k.unit, -kLowest);
  k.half_slack = std::min(kSlack2 / 2 / k.unit, -kLowest);
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
