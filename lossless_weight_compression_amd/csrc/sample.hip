// sample.hip -- temperature, top-k, top-p and min-p on rows of logits, the next
// token from a given random number, and the filtered probabilities
// (enc_sample).
//
// With x = l / T and the tokens of a row in the order of their logits
// (descending, ties by index), each filter keeps a front part of the order, so
// what is kept ends at one token: the cut. Nothing is sorted. A first pass puts
// every token into one of 768 bins of 1/16 in x below the row's greatest, counts
// them and sums their weights e^x; cumulative counts and sums name the bins in
// which the cuts lie; only those bins' tokens (some hundred) are gathered, by a
// second pass, and selected from.
//
// Sums: bin edges are whole multiples of 1/16 in x itself, not below the
// greatest, so that segments of a row, which do not know the row's greatest,
// count into the same bins. Within a bin a weight is taken relative to the
// bin's lower edge, 1 <= w < 1.065, and held as a whole number of 2^-32: sums in a bin
// are exact in any order (in fp64 too, for 2^20 tokens, so that borders between
// equal logits are met exactly), and a count and a sum fit one 64-bit word of
// LDS. Across bins sums are fp64, always in the same order. The borders between
// tokens are finer than fp32: in 128256 tokens a cumulative sum that is off by
// 1e-8 draws another token once in a thousand calls; here it is some 1e-12.
//
// Steps, each a launch: k_scan (rows x segments), k_plan (rows), k_collect (rows
// x segments with something to gather), k_resolve (rows; the cut, the draw),
// k_probs (rows x segments). Where more than 4096 tokens lie in a cut's bins
// (many equal logits, a high temperature), k_resolve reads the row itself.
//
// Bound: for a few rows the chain of launches and, in each, the way from loads over
// an exchange to stores; for many rows the instructions for a token (17 in the
// first pass) and its LDS atomic, not the bytes. Measured, 128256 tokens: 1 row 28
// us (scan 4.8, plan 9.4, collect 4.0, resolve 12.2), 64 rows of BF16 with ties 49
// (10.3, 11.1, 7.7, 19.7), 256 rows 94 (32.9, 11.0, 25.0, 24.8; one read of the logits at
// a copy's rate is 26). Probabilities of 96 rows of 32000: 41 to 44 us for FP32, BF16
// and FP16 in any pair, 45 to 46 from 16-bit logits to FP32, which are stored one by
// one. Where k_resolve reads the row, by the passes of each cut: one row of equal
// logits 711 us with top-p, 1256 with top-k of 40000 too; logits of unit spread, which
// reach it with both, 257 (BF16 433), 64 rows 355 (454).
#include "step_common.h"

#include "group_math.h"

#include <algorithm>
#include <type_traits>

namespace enc {
namespace {

typedef unsigned long long u64;
constexpr uint32_t kBins = kSampleBins, kList = kSampleList, kWide = 1024;
constexpr double kUnit = 1.0 / 4294967296.0;   // 2^-32
constexpr u64 kOne = 1ull << 32, kSumMask = (1ull << 49) - 1;
constexpr uint32_t kNoBin = ~0u;

// Keys: greater for tokens earlier in the order; never 0.
__device__ __forceinline__ u64 key_of(float l, uint32_t i) {
  const uint32_t u = __float_as_uint(l + 0.f);   // -0 counts as 0
  return (u64)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float logit_of(u64 key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint32_t index_of(u64 key) { return ~(uint32_t)key; }
// NaN and -infinity are never kept.
__device__ __forceinline__ bool counts(float l) { return l > -__builtin_inff(); }

// Place in units of 1/16 of x, rounded to a multiple of 2^-30 (2^-35 of a weight):
// logits that differ by less, around 0 on both sides of a bin's edge, weigh the
// same to the bit. +infinity lies above everything finite.
__device__ __forceinline__ double place_of(float l, double r16) {
  constexpr double kRound = 6291456.0;   // 3 2^21: one unit in its last place is 2^-30
  return l == __builtin_inff() ? 1e300 : fma((double)l, r16, kRound) - kRound;
}
// e^(f / 16) - 1 for f = n 2^-30 < 1 in units of 2^-32, rounded (the next term of
// the series is below 2^-40).
__device__ __forceinline__ uint32_t excess_of(uint32_t n) {
  constexpr double z = 1.0 / 17179869184.0, one = 4294967296.0;   // 2^-34: f / 16 is n z
  const double x = (double)n;
  double s = one * z * z * z * z * z * z / 720.0;
  s = fma(s, x, one * z * z * z * z * z / 120.0);
  s = fma(s, x, one * z * z * z * z / 24.0);
  s = fma(s, x, one * z * z * z / 6.0);
  s = fma(s, x, one * z * z / 2.0);
  s = fma(s, x, one * z);
  // the low bits of 2^52 + m are m
  return (uint32_t)__double_as_longlong(fma(s, x, 4503599627370496.0));
}

// e^(-i / 16), a bin's lower edge relative to the first bin's: whole powers of e
// times sixteenths (rounded to fp64 each).
__device__ const double kWholes[48] = {
    1.0, 0.36787944117144233, 0.1353352832366127, 0.049787068367863944,
    0.01831563888873418, 0.006737946999085467, 0.0024787521766663585, 0.0009118819655545162,
    0.00033546262790251185, 0.00012340980408667956, 4.5399929762484854e-05, 1.670170079024566e-05,
    6.14421235332821e-06, 2.2603294069810542e-06, 8.315287191035679e-07, 3.059023205018258e-07,
    1.1253517471925912e-07, 4.139937718785167e-08, 1.522997974471263e-08, 5.602796437537268e-09,
    2.061153622438558e-09, 7.582560427911907e-10, 2.7894680928689246e-10, 1.026187963170189e-10,
    3.775134544279098e-11, 1.3887943864964021e-11, 5.109089028063325e-12, 1.8795288165390832e-12,
    6.914400106940203e-13, 2.543665647376923e-13, 9.357622968840175e-14, 3.442477108469977e-14,
    1.2664165549094176e-14, 4.658886145103398e-15, 1.713908431542013e-15, 6.305116760146989e-16,
    2.3195228302435696e-16, 8.533047625744066e-17, 3.1391327920480296e-17, 1.1548224173015786e-17,
    4.248354255291589e-18, 1.5628821893349888e-18, 5.74952226429356e-19, 2.1151310375910805e-19,
    7.781132241133797e-20, 2.8625185805493937e-20, 1.0530617357553812e-20, 3.873997628687187e-21};
__device__ const double kParts[16] = {
    1.0, 0.9394130628134758, 0.8824969025845955, 0.8290291181804004,
    0.7788007830714049, 0.7316156289466418, 0.6872892787909722, 0.645648526427892,
    0.6065306597126334, 0.569782824730923, 0.5352614285189903, 0.5028315779709409,
    0.4723665527410147, 0.44374731008107987, 0.4168620196785084, 0.391605626676799};
static_assert(kBins == 48 * 16, "the tables cover the bins");
__device__ __forceinline__ void fill_edges(double *edges) {   // in LDS
  for (uint32_t i = threadIdx.x; i < kBins; i += blockDim.x) edges[i] = kWholes[i >> 4] * kParts[i & 15];
}

// A token's bin below `edge` (kBins or more: none) and excess. Where the first
// bin's place is below 2^20 in size, both are read off the bits of the rounded
// sum 3 2^21 + place: 30 bits of fraction, then the whole number under an exponent
// that is the same for all. Logits far below (NaN and -infinity among them) are
// raised to one that is in no bin.
struct Places {
  double r16, edge;
  float lowest;
  uint32_t first;      // the first bin's bits from the 30th on
  bool near_;
  __device__ __forceinline__ Places(double r, double e) : r16(r), edge(e) {
    near_ = fabs(e) < 1048576.0 && r > 1e-30;
    lowest = near_ ? (float)(-2000000.0 / r) : 0.f;   // place above -2^21
    first = (uint32_t)((u64)__double_as_longlong(6291456.0 + (near_ ? e : 0.0)) >> 30);
  }
  template <bool NEAR> __device__ __forceinline__ uint32_t bin_of(float l, uint32_t &excess) const {
    if constexpr (NEAR) {
      const u64 bits = (u64)__double_as_longlong(fma((double)fmaxf(l, lowest), r16, 6291456.0));
      excess = excess_of((uint32_t)bits & 0x3FFFFFFFu);
      return first - (uint32_t)(bits >> 30);
    } else {
      const double t = place_of(l, r16), at = floor(t), below = edge - at;
      if (!counts(l) || !(below < (double)kBins)) return kBins;
      excess = excess_of((uint32_t)((t - at) * 1073741824.0));   // whole: t is a multiple of 2^-30, or of 1
      return (uint32_t)below;
    }
  }
  __device__ __forceinline__ uint32_t bin_of(float l, uint32_t &excess) const {
    return near_ ? bin_of<true>(l, excess) : bin_of<false>(l, excess);
  }
};

struct Setting {
  double r16;        // 16 / temperature
  double top_p, min_p;
  uint32_t top_k;    // 0: all
  bool first;        // only the first of the order
};
__device__ __forceinline__ Setting setting_of(const enc_sample_args &a, uint32_t row) {
  const uint32_t i = row / a.rows_per_setting;
  Setting s;
  const float t = a.d_temperature ? a.d_temperature[i] : 1.f;
  s.first = !(t > 0.f);
  s.r16 = s.first ? 16.0 : 16.0 / (double)t;
  const int32_t k = a.d_top_k ? a.d_top_k[i] : 0;
  s.top_k = k > 0 && (uint32_t)k < a.vocab ? (uint32_t)k : 0;
  const float p = a.d_top_p ? a.d_top_p[i] : 1.f;
  s.top_p = p < 1.f ? (double)p : 1.0;
  const float m = a.d_min_p ? a.d_min_p[i] : 0.f;
  s.min_p = m > 0.f ? (double)m : 0.0;
  s.first = s.first || s.top_k == 1 || s.top_p <= 0.0 || s.min_p > 1.0;
  return s;
}

// ---- a row in 16-byte pieces: piece boundaries are those of memory, so element
// i of the row is place i + head of the row's pieces
template <typename T> constexpr uint32_t kPiece = 16 / sizeof(T);
template <typename T> __device__ __forceinline__ uint32_t head_of(const T *row) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T);
}
template <typename T> __device__ __forceinline__ float value_at(const T *row, uint32_t i) { return (float)row[i]; }

template <typename T>
__device__ __forceinline__ uint4 load_piece(const T *row, uint32_t head, uint32_t vocab, uint32_t at) {
  constexpr uint32_t E = kPiece<T>;
  if (at >= head && at + E <= head + vocab) return *reinterpret_cast<const uint4 *>(row + ((int64_t)at - head));
  uint32_t w[4];
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) {   // -infinity where there is no element
    if constexpr (sizeof(T) == 4) {
      const uint32_t v = at + e;
      w[e] = v >= head && v < head + vocab ? reinterpret_cast<const uint32_t *>(row)[v - head] : 0xFF800000u;
    } else {
      constexpr uint32_t kNone = std::is_same<T, __bf16>::value ? 0xFF80u : 0xFC00u;
      const uint32_t v = at + 2 * e;
      const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
      const uint32_t lo = v >= head && v < head + vocab ? p[v - head] : kNone;
      const uint32_t hi = v + 1 >= head && v + 1 < head + vocab ? p[v + 1 - head] : kNone;
      w[e] = lo | hi << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T> __device__ __forceinline__ void values_of(uint4 piece, float (&x)[kPiece<T>]) {
  const uint32_t w[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
  for (uint32_t e = 0; e < kPiece<T>; ++e) {
    if constexpr (sizeof(T) == 4)
      x[e] = __uint_as_float(w[e]);
    else
      x[e] = half_of<T>(w[e >> 1], e & 1);
  }
}

__device__ __forceinline__ u64 wave_max(u64 v) {
  for (uint32_t o = 32; o; o >>= 1) {
    const u64 w = __shfl_xor(v, o);
    v = w > v ? w : v;
  }
  return v;
}

template <typename V> __device__ __forceinline__ V wave_total(V v) {
  for (uint32_t o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <typename V> __device__ __forceinline__ V wave_scan(V v) {   // inclusive
  const uint32_t lane = threadIdx.x & 63;
  for (uint32_t o = 1; o < 64; o <<= 1) {
    const V w = __shfl_up(v, o);
    if (lane >= o) v += w;
  }
  return v;
}
// Inclusive scan over a workgroup of kWide; `side` has room for 16 and is free
// again after the call's last barrier.
template <typename V> __device__ __forceinline__ V group_scan(V v, V *side) {
  v = wave_scan(v);
  const uint32_t wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 63) side[wave] = v;
  __syncthreads();
  V before = 0;
#pragma unroll
  for (uint32_t w = 0; w < kWide / 64; ++w) {   // all read at once
    const V other = side[w];
    if (w < wave) before += other;
  }
  return before + v;
}

// ---- first pass: a segment's greatest key, and its bins
template <typename T, uint32_t NT, uint32_t NV>
__global__ __launch_bounds__(NT) void k_scan(SampleKernelArgs k) {
  constexpr uint32_t E = kPiece<T>, S = NT * NV * E;
  const enc_sample_args &a = k.a;
  __shared__ u64 bins[kBins];
  __shared__ float tops[NT / 64];
  __shared__ uint32_t last, lowest;
  const uint32_t tid = threadIdx.x, r = blockIdx.x / k.segments, seg = blockIdx.x - r * k.segments;
  const uint32_t row = k.row0 + r;
  const T *l = static_cast<const T *>(a.d_logits) + (uint64_t)row * a.logits_row;
  const uint32_t head = head_of(l);
  uint4 piece[NV];
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) piece[j] = load_piece(l, head, a.vocab, seg * S + (j * NT + tid) * E);
  const Setting set = setting_of(a, row);
  for (uint32_t i = tid; i < kBins; i += NT) bins[i] = 0;
  if (tid == 0) last = 0, lowest = ~0u;

  float best = -__builtin_inff();   // (NaN is passed over)
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) {
    float x[E];
    values_of<T>(piece[j], x);
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) best = fmaxf(best, x[e]);
  }
  for (uint32_t o = 32; o; o >>= 1) best = fmaxf(best, __shfl_xor(best, o));
  if ((tid & 63) == 0) tops[tid >> 6] = best;
  __syncthreads();
  for (uint32_t w = 0; w < NT / 64; ++w) best = fmaxf(best, tops[w]);
  // the first token that has it: only asked for where no other is kept
  if (set.first && counts(best)) {
    uint32_t at = ~0u;
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      float x[E];
      values_of<T>(piece[j], x);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e)
        if (x[e] == best) at = min(at, seg * S + (j * NT + tid) * E + e - head);
    }
    if (at != ~0u) atomicMin(&lowest, at);
    __syncthreads();
  }
  const u64 top = counts(best) ? key_of(best, set.first ? lowest : 0u) : 0ull;
  SampleSegment *out = k.segs + (uint64_t)r * k.segments + seg;
  if (tid == 0) {
    out->top = top;
    out->bins = 0;
  }
  if (top == 0 || set.first) return;   // nothing in it, or nothing but the first is asked for
  const double edge = floor(place_of(logit_of(top), set.r16));
  const Places places(set.r16, edge);
  const auto fill = [&](auto near_) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      float x[E];
      values_of<T>(piece[j], x);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        uint32_t excess;
        const uint32_t bin = places.bin_of<decltype(near_)::value>(x[e], excess);
        if (bin < kBins) atomicAdd(&bins[bin], (1ull << 49) + excess);
      }
    }
  };
  if (places.near_)
    fill(std::true_type{});
  else
    fill(std::false_type{});
  __syncthreads();
  u64 *dst = k.bins + ((uint64_t)r * k.segments + seg) * kBins;
  uint32_t used = 0;
  u64 mine[(kBins + NT - 1) / NT];
#pragma unroll
  for (uint32_t j = 0; j < (kBins + NT - 1) / NT; ++j) {
    const uint32_t i = tid + j * NT;
    mine[j] = i < kBins ? bins[i] : 0;
    if (mine[j]) used = i + 1;
  }
  for (uint32_t o = 32; o; o >>= 1) used = max(used, (uint32_t)__shfl_xor((int)used, o));
  if ((tid & 63) == 0) atomicMax(&last, used);   // (64 lanes with values of their own would go one by one)
  __syncthreads();
  used = last;
#pragma unroll
  for (uint32_t j = 0; j < (kBins + NT - 1) / NT; ++j)
    if (tid + j * NT < used) dst[tid + j * NT] = mine[j];
  if (tid == 0) {
    out->edge = edge;
    out->bins = used;
  }
}

// ---- per row: the bins of all segments, and where the cuts lie
__global__ __launch_bounds__(kWide) void k_plan(SampleKernelArgs k) {
  const enc_sample_args &a = k.a;
  __shared__ u64 tops[kWide / 64];
  __shared__ double sums[kBins], side[kWide / 64];
  __shared__ uint32_t numbers[kBins], side_n[kWide / 64];
  __shared__ uint32_t k_bin, p_low, p_high;
  __shared__ uint32_t starts[kSampleSegments], used[kSampleSegments], gathered[kSampleSegments];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = blockIdx.x, row = k.row0 + r;
  SampleSegment *segs = k.segs + (uint64_t)r * k.segments;
  const Setting set = setting_of(a, row);
  SampleRow &out = k.rows[r];
  const uint32_t segments = k.segments;

  // (a segment to a thread: there are at most as many)
  u64 top = 0;
  double my_edge = 0.0;
  uint32_t my_used = 0;
  if (tid < segments) {
    top = segs[tid].top;
    my_edge = segs[tid].edge;
    my_used = segs[tid].bins;
  }
  top = wave_max(top);
  if (lane == 0) tops[wave] = top;
  if (tid == 0) k_bin = p_low = p_high = kBins - 1;
  __syncthreads();
  for (uint32_t w = 0; w < kWide / 64; ++w) top = max(top, tops[w]);
  const double t_max = place_of(logit_of(top), set.r16), edge = floor(t_max);
  if (tid == 0) {
    out.edge = edge;
    out.r16 = set.r16;
    out.top = top;
    out.n = 0;
    out.cut_bin = 0;
    out.tau = top;
    // one token alone: its weight, relative to its bin's lower edge
    out.z = top == 0 ? 0.0 : 1.0 + (double)excess_of((uint32_t)((t_max - edge) * 1073741824.0)) * kUnit;
    out.state = top == 0 ? kSampleEmpty : kSampleFirst;
  }
  if (top == 0 || set.first) return;
  if (tid < segments) {
    const double by = edge - my_edge;   // (an empty segment's edge is nothing)
    const bool any = my_used && by < (double)kBins;
    starts[tid] = any ? (uint32_t)by : 0u;
    used[tid] = any ? my_used : 0u;
  }
  __syncthreads();

  u64 sum = 0;
  uint32_t number = 0;
  if (tid < kBins) {
    const u64 *bins = k.bins + (uint64_t)r * segments * kBins;
#pragma unroll 8
    for (uint32_t s = 0; s < segments; ++s) {
      const uint32_t at = tid - starts[s];   // wraps where the segment has no such bin
      const bool has = at < used[s];
      const u64 v = bins[(uint64_t)s * kBins + (has ? at : 0)];
      number += has ? (uint32_t)(v >> 49) : 0;
      sum += has ? v & kSumMask : 0;
    }
  }
  const double mass =
      tid < kBins ? ((double)number + (double)sum * kUnit) * (kWholes[tid >> 4] * kParts[tid & 15]) : 0.0;
  const double upto = group_scan(mass, side);
  const uint32_t n_upto = group_scan(number, side_n);
  if (tid < kBins) {
    sums[tid] = upto;
    numbers[tid] = n_upto;
    k.sums[(uint64_t)r * kBins + tid] = upto;
  }
  __syncthreads();
  // The bin that a count or a sum is reached in. Counts grow, so that test is true
  // once; sums of neighbouring bins are taken in different orders and may fall by a
  // rounding, so the first bin counts.
  if (set.top_k && tid < kBins && n_upto >= set.top_k && n_upto - number < set.top_k) k_bin = tid;
  __syncthreads();
  const uint32_t kb = k_bin;
  const bool k_part = set.top_k && numbers[kb] > set.top_k;
  if (set.top_p < 1.0 && tid < kBins) {
    const double low = set.top_p * (k_part ? kb ? sums[kb - 1] : 0.0 : sums[kb]), high = set.top_p * sums[kb];
    const uint64_t lows = __ballot(upto >= low), highs = __ballot(upto >= high);
    if (lane == 0 && lows) atomicMin(&p_low, tid + __builtin_ctzll(lows));
    if (lane == 0 && highs) atomicMin(&p_high, tid + __builtin_ctzll(highs));
  }
  __syncthreads();
  uint32_t bk = k_part ? kb : kNoBin, lo = set.top_p < 1.0 ? p_low : kNoBin, hi = set.top_p < 1.0 ? min(p_high, kb) : kb;
  if (lo != kNoBin) lo = min(lo, hi);
  double t_min = -1e308;
  uint32_t bm = kNoBin;
  if (set.min_p > 0.0) {
    t_min = t_max + 16.0 * log(set.min_p);
    const double below = edge - floor(t_min);
    if (below < (double)kBins) bm = (uint32_t)below;
    if (bm != kNoBin && bm > min(hi, kb)) bm = kNoBin;                   // another filter ends before it
    if (bm != kNoBin && bm < min(bk, lo) && (lo != kNoBin || bk != kNoBin)) bk = lo = kNoBin;   // it ends before the others
    if (bm != kNoBin && bk == kNoBin && lo == kNoBin) hi = bm;
  }
  // tokens to gather, and every segment's place in the list
  const auto wanted = [&](uint32_t i) { return i == bk || i == bm || (lo != kNoBin && i >= lo && i <= hi); };
  uint32_t total = 0;
  if (bk != kNoBin || bm != kNoBin || lo != kNoBin) {
    uint32_t mine = 0;
    if (tid < kBins && wanted(tid)) mine = number;
    total = group_scan(mine, side_n);
    __syncthreads();
    if (tid == kWide - 1) side_n[0] = total;
    __syncthreads();
    total = side_n[0];
    if (total <= kList) {
      // a wave counts a segment's wanted bins; then a scan over the segments
      for (uint32_t s = wave; s < segments; s += kWide / 64) {
        const u64 *bins = k.bins + ((uint64_t)r * segments + s) * kBins;
        uint32_t c = 0;
#pragma unroll
        for (uint32_t i0 = 0; i0 < kBins; i0 += 64) {
          const uint32_t i = i0 + lane;
          const bool has = i < used[s] && i + starts[s] < kBins && wanted(i + starts[s]);
          const u64 v = bins[has ? i : 0];
          c += has ? (uint32_t)(v >> 49) : 0;
        }
        c = wave_incl_scan(c);
        if (lane == 63) gathered[s] = c;
      }
      __syncthreads();
      const uint32_t c = tid < segments ? gathered[tid] : 0;
      const uint32_t incl = group_scan(c, side_n);
      if (tid < segments) {
        segs[tid].n = c;
        segs[tid].first = incl - c;
      }
    }
  }
  if (tid == 0) {
    out.bk = bk;
    out.lo = lo;
    out.hi = hi;
    out.bm = bm;
    out.kb = kb;
    out.rank = k_part ? set.top_k - (kb ? numbers[kb - 1] : 0) : 0;   // the last kept one's, from 1
    out.top_p = set.top_p;
    out.t_min = t_min;
    out.n = total;
    out.bk_n = k_part ? numbers[kb] - (kb ? numbers[kb - 1] : 0) : 0;
    out.lo_n = lo != kNoBin && lo == hi ? numbers[lo] - (lo ? numbers[lo - 1] : 0) : 0;
    out.cut_bin = hi;   // where no list is needed: a whole bin ends what is kept
    out.tau = 0;
    out.z = sums[hi];
    out.state = total == 0 ? kSampleWhole : total <= kList ? kSampleListed : kSampleRead;
  }
}

// ---- second pass: the tokens of the cuts' bins
template <typename T, uint32_t NT, uint32_t NV>
__global__ __launch_bounds__(NT) void k_collect(SampleKernelArgs k) {
  constexpr uint32_t E = kPiece<T>, S = NT * NV * E;
  const enc_sample_args &a = k.a;
  __shared__ uint32_t filled;
  const uint32_t tid = threadIdx.x, r = blockIdx.x / k.segments, seg = blockIdx.x - r * k.segments;
  const SampleRow &w = k.rows[r];
  if (w.state != kSampleListed) return;
  const SampleSegment &me = k.segs[(uint64_t)r * k.segments + seg];
  if (!me.bins || !me.n) return;
  const T *l = static_cast<const T *>(a.d_logits) + (uint64_t)(k.row0 + r) * a.logits_row;
  const uint32_t head = head_of(l);
  uint4 piece[NV];
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) piece[j] = load_piece(l, head, a.vocab, seg * S + (j * NT + tid) * E);
  if (tid == 0) filled = 0;
  __syncthreads();
  const uint32_t bk = w.bk, lo = w.lo, hi = w.hi, bm = w.bm;
  const Places places(w.r16, w.edge);
  const uint32_t n = me.n;
  SampleToken *dst = k.list + (uint64_t)r * kList + me.first;
  const auto gather = [&](auto near_) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      float x[E];
      values_of<T>(piece[j], x);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        uint32_t excess;
        const uint32_t i = places.bin_of<decltype(near_)::value>(x[e], excess);
        if (i < kBins && (i == bk || i == bm || (i >= lo && i <= hi))) {   // (without lo nothing is as large)
          const uint32_t slot = atomicAdd(&filled, 1u);   // any order: what is selected does not depend on it
          if (slot < n) dst[slot] = SampleToken{key_of(x[e], seg * S + (j * NT + tid) * E + e - head), (u64)i << 40 | excess};
        }
      }
    }
  };
  if (places.near_)
    gather(std::true_type{});
  else
    gather(std::false_type{});
}

// ---- per row: the cuts among the gathered tokens, then the draw

constexpr uint32_t kFew = 64;   // few enough for one wave, a token to a lane
struct Select {
  u64 keys[kFew], weights[kFew];
  u64 sum[256];         // of a digit's values
  uint32_t number[256];
  u64 any, every, tau, upto, skipped_sum;
  uint32_t filled, digit, skipped, left;
};

// Tokens of a row: those gathered, or the row itself. f(key, bin, excess).
template <typename T> struct Tokens {
  const SampleToken *list;   // in LDS
  uint32_t n;
  const T *row;              // instead, if not NULL
  uint32_t vocab;
  double r16, edge;
  template <typename F> __device__ __forceinline__ void each(F f) const {
    if (!row) {
      for (uint32_t i = threadIdx.x; i < n; i += kWide)
        f(list[i].key, (uint32_t)(list[i].at >> 40), list[i].at & ((1ull << 40) - 1));
    } else {
      const Places places(r16, edge);
#pragma unroll 4
      for (uint32_t i = threadIdx.x; i < vocab; i += kWide) {
        const float x = value_at(row, i);
        uint32_t excess;
        const uint32_t bin = places.bin_of(x, excess);
        if (bin < kBins) f(key_of(x, i), bin, (u64)excess);
      }
    }
  }
};

// The key of the token of a bin, in the order, at which the count reaches `rank`
// (from 1), or, with rank 0, the weights' sum reaches `need` (in bin units); the
// bin's last token if neither does. `left`: how many the bin has. First a digit
// of the excess, which spreads a bin's tokens, then, where many are equal, digits
// of the key from its highest bit that differs, until a wave has a lane for each.
// `upto`: the bin's weights from its first token to that one, in units of 2^-32.
template <typename T>
__device__ u64 select(const Tokens<T> &all, uint32_t bin, uint32_t left, uint32_t rank, double need, Select &s, u64 &upto) {
  const uint32_t tid = threadIdx.x, lane = tid & 63;
  u64 low = 0, high = ~0ull;   // keys still in question
  uint32_t qd = kNoBin;        // their excess' first digit
  uint32_t skipped = 0;        // tokens and weights before them
  u64 skipped_sum = 0;
  const auto live = [&](u64 key, uint32_t i, u64 q) {
    return i == bin && key >= low && key <= high && (qd == kNoBin || (uint32_t)(q >> 21) == qd);
  };
  for (uint32_t round = 0; left > kFew; ++round) {
    const bool by_excess = round == 0;
    uint32_t shift = 0;
    u64 common = 0;
    __syncthreads();
    if (tid < 256) s.sum[tid] = 0, s.number[tid] = 0;
    if (tid == 0) s.any = 0, s.every = ~0ull;
    __syncthreads();
    if (!by_excess) {   // where they differ
      u64 any = 0, every = ~0ull;
      all.each([&](u64 key, uint32_t i, u64 q) {
        if (!live(key, i, q)) return;
        any |= key;
        every &= key;
      });
      for (uint32_t o = 32; o; o >>= 1) {
        any |= __shfl_xor(any, o);
        every &= __shfl_xor(every, o);
      }
      if (lane == 0 && any) {
        atomicOr(&s.any, any);
        atomicAnd(&s.every, every);
      }
      __syncthreads();
      common = s.every;
      const uint32_t top_bit = 63 - __clzll((long long)(s.any & ~common));   // keys are distinct: some bit differs
      shift = top_bit >= 7 ? top_bit - 7 : 0;
    }
    all.each([&](u64 key, uint32_t i, u64 q) {
      if (!live(key, i, q)) return;
      const uint32_t d = by_excess ? (uint32_t)(q >> 21) : (uint32_t)(key >> shift) & 255u;
      atomicAdd(&s.number[d], 1u);
      atomicAdd(&s.sum[d], kOne + q);
    });
    __syncthreads();
    if (tid < 64) {   // digits from the highest down, four to a lane
      uint32_t n4 = 0;
      u64 m4 = 0;
      for (uint32_t e = 0; e < 4; ++e) n4 += s.number[255 - 4 * lane - e], m4 += s.sum[255 - 4 * lane - e];
      uint32_t n_at = skipped + wave_scan(n4) - n4;
      u64 m_at = skipped_sum + wave_scan(m4) - m4;
      uint32_t hit = kNoBin, last = kNoBin;
      for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t d = 255 - 4 * lane - e;
        if (!s.number[d]) continue;
        last = d;
        const bool reached = rank ? n_at + s.number[d] >= rank : (double)(m_at + s.sum[d]) * kUnit >= need;
        if (reached && hit == kNoBin) hit = d;
        if (hit == kNoBin) n_at += s.number[d], m_at += s.sum[d];
      }
      const u64 hits = __ballot(hit != kNoBin), lasts = __ballot(last != kNoBin);
      // the first lane that reaches it; if none does (rounding), the last token
      const int from = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(lasts);
      const uint32_t d = __builtin_amdgcn_readlane(hits ? hit : last, from);
      if (!hits) {   // everything before the last digit is passed
        n_at = skipped, m_at = skipped_sum;
        for (uint32_t e = 255; e > d; --e) n_at += s.number[e], m_at += s.sum[e];
      } else {
        n_at = __builtin_amdgcn_readlane(n_at, from);
        m_at = (u64)(uint32_t)__builtin_amdgcn_readlane((uint32_t)m_at, from) |
               (u64)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(m_at >> 32), from) << 32;
      }
      if (lane == 0) s.digit = d, s.skipped = n_at, s.skipped_sum = m_at, s.left = s.number[d];
    }
    __syncthreads();
    skipped = s.skipped;
    skipped_sum = s.skipped_sum;
    left = s.left;
    if (by_excess) {
      qd = s.digit;
    } else {
      const u64 same = shift + 8 < 64 ? common >> (shift + 8) << (shift + 8) : 0;   // bits above the digit
      low = same | (u64)s.digit << shift;
      high = low | ((1ull << shift) - 1);
    }
  }
  __syncthreads();
  if (tid == 0) s.filled = 0;
  __syncthreads();
  all.each([&](u64 key, uint32_t i, u64 q) {
    if (!live(key, i, q)) return;
    const uint32_t slot = atomicAdd(&s.filled, 1u);
    if (slot < kFew) s.keys[slot] = key, s.weights[slot] = kOne + q;
  });
  __syncthreads();
  if (tid < 64) {
    const uint32_t n = min(s.filled, kFew);
    const u64 key = lane < n ? s.keys[lane] : 0, weight = lane < n ? s.weights[lane] : 0;
    uint32_t number = skipped;
    u64 sum = skipped_sum;
    for (uint32_t j = 0; j < n; ++j) {
      const u64 other = s.keys[j], w = s.weights[j];
      if (other > key) ++number, sum += w;
    }
    // not yet reached before this one: the least such key is the one
    const bool kept = lane < n && (rank ? number < rank : (double)sum * kUnit < need);
    u64 least = kept ? key : ~0ull;
    for (uint32_t o = 32; o; o >>= 1) {
      const u64 w = __shfl_xor(least, o);
      least = w < least ? w : least;
    }
    if (kept && key == least) s.tau = key, s.upto = sum + weight;
    if (lane == 0 && least == ~0ull) s.tau = ~0ull, s.upto = skipped_sum;
  }
  __syncthreads();
  upto = s.upto;
  return s.tau;
}

// ROUNDS: 64 tokens at a time, of a sixteenth of a segment.
template <typename T, uint32_t ROUNDS>
__global__ __launch_bounds__(kWide) void k_resolve(SampleKernelArgs k) {
  const enc_sample_args &a = k.a;
  __shared__ SampleToken list[kList];
  __shared__ Select pick;
  __shared__ double sums[kBins], edges[kBins], side[kWide / 64], masses[kWide];
  __shared__ u64 parts[kSampleSegments];
  __shared__ u64 part, lowest;
  __shared__ uint32_t chosen, counted;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = blockIdx.x, row = k.row0 + r;
  SampleRow &w = k.rows[r];
  const uint32_t state = w.state;
  const u64 top = w.top;
  if (state == kSampleEmpty || state == kSampleFirst) {
    if (tid == 0) {
      if (a.d_token) a.d_token[row] = state == kSampleEmpty ? -1 : (int32_t)index_of(top);
    }
    return;
  }
  const T *l = static_cast<const T *>(a.d_logits) + (uint64_t)row * a.logits_row;
  const uint32_t head = head_of(l);
  const double r16 = w.r16, edge = w.edge;
  const uint32_t listed = w.n;
  constexpr uint32_t kShift = ROUNDS == 4 ? 12 : 14;   // of a segment of 1024 ROUNDS
  static_assert(1u << kShift == 1024 * ROUNDS, "a segment is 1024 times the rounds");
  uint32_t cut = w.cut_bin;
  u64 tau = 0;
  double z = w.z;
  fill_edges(edges);
  if (state != kSampleWhole) {
    Tokens<T> all;
    all.list = list;
    all.n = state == kSampleListed ? listed : 0;
    all.row = state == kSampleListed ? nullptr : l;
    all.vocab = a.vocab;
    all.r16 = r16;
    all.edge = edge;
    for (uint32_t i = tid; i < all.n; i += kWide) list[i] = k.list[(uint64_t)r * kList + i];
    if (tid < kBins) sums[tid] = k.sums[(uint64_t)r * kBins + tid];
    for (uint32_t s = tid; s < k.segments; s += kWide) parts[s] = 0;
    __syncthreads();
    const uint32_t bk = w.bk, lo = w.lo, bm = w.bm, kb = w.kb;
    // tokens of a bin that top-p may cut: known where there is one such bin
    const auto count_in = [&](uint32_t bin) {
      if (bin == w.hi && lo == w.hi) return w.lo_n;
      __syncthreads();
      if (tid == 0) counted = 0;
      __syncthreads();
      uint32_t n = 0;
      all.each([&](u64, uint32_t i, u64) { n += i == bin; });
      n = wave_total(n);
      if (lane == 0 && n) atomicAdd(&counted, n);
      __syncthreads();
      return counted;
    };
    const auto upto = [&](uint32_t bin) { return bin ? sums[bin - 1] : 0.0; };
    const auto unit_of = [&](uint32_t bin) { return edges[bin]; };
    cut = kb;
    double kept = sums[kb];
    u64 in_cut = 0;   // kept weights of the cut's bin, where tau says which
    if (bk != kNoBin) {
      tau = select(all, bk, w.bk_n, w.rank, 0.0, pick, in_cut);
      kept = upto(bk) + (double)in_cut * kUnit * unit_of(bk);
    }
    if (lo != kNoBin) {
      const double goal = w.top_p * kept;
      uint32_t b = lo;
      while (b < w.hi && sums[b] < goal) ++b;
      // (never less than the first token, whatever the rounding)
      u64 in_b;
      const u64 at = select(all, b, count_in(b), 0, fmax((goal - upto(b)) / unit_of(b), 1e-300), pick, in_b);
      if (b < cut || at > tau) tau = at, in_cut = in_b;
      cut = b;
    }
    if (bm != kNoBin && bm <= cut) {
      if (tid == 0) lowest = ~0ull, part = 0;   // nothing of the bin, if none is great enough
      __syncthreads();
      const double t_min = w.t_min;
      u64 sum = 0, least = ~0ull;
      all.each([&](u64 key, uint32_t i, u64 q) {
        if (i != bm || place_of(logit_of(key), r16) < t_min) return;
        least = min(least, key);
        sum += kOne + q;
      });
      sum = wave_total(sum);
      least = ~wave_max(~least);
      if (lane == 0 && sum) {
        atomicAdd(&part, sum);
        atomicMin(&lowest, least);
      }
      __syncthreads();
      if (bm < cut || lowest > tau) tau = lowest, in_cut = part;
      cut = bm;
    }
    // (tau 0: a whole bin, which only a filter that ends with it leaves)
    z = tau ? upto(cut) + (double)in_cut * kUnit * unit_of(cut) : sums[cut];
    if (tid == 0) {
      w.cut_bin = cut;
      w.tau = tau;
      w.z = z;
    }
    if (state == kSampleRead && tau && a.d_token) {   // each segment's part of the cut's bin
      __syncthreads();
      all.each([&](u64 key, uint32_t i, u64 q) {
        if (i == cut && key >= tau) atomicAdd(&parts[(index_of(key) + head) >> kShift], kOne + q);
      });
    }
  }
  if (!a.d_token) return;

  // the segments' kept weights: bins above the cut, and of its bin what is above tau
  __syncthreads();
  // (several waves to a segment where there are few)
  const uint32_t ways = k.segments > 8 ? 1 : k.segments > 4 ? 2 : k.segments > 2 ? 4 : 8;
  for (uint32_t unit = wave; unit < k.segments * ways; unit += kWide / 64) {
    const uint32_t s = unit / ways, way = unit - s * ways;
    const SampleSegment &seg = k.segs[(uint64_t)r * k.segments + s];
    const u64 *bins = k.bins + ((uint64_t)r * k.segments + s) * kBins;
    const uint32_t n = seg.bins;
    const double by = edge - seg.edge;
    double m = 0.0;
    if (n && by < (double)kBins) {
      const uint32_t d = (uint32_t)by, end = min(n, cut + 1 > d ? cut + 1 - d : 0u);
#pragma unroll 4
      for (uint32_t i = 64 * way + lane; i < end; i += 64 * ways) {
        const u64 v = bins[i];
        m += d + i < cut || !tau ? ((double)(v >> 49) + (double)(v & kSumMask) * kUnit) * edges[d + i] : 0.0;
      }
    }
    m = wave_total(m);
    if (tau) {
      u64 in_cut = state == kSampleRead && way == 0 ? parts[s] : 0;
      if (state == kSampleListed) {
#pragma unroll 4
        for (uint32_t i = 64 * way + lane; i < listed; i += 64 * ways) {
          const SampleToken t = list[i];
          const bool mine_too = (uint32_t)(t.at >> 40) == cut && t.key >= tau && (index_of(t.key) + head) >> kShift == s;
          in_cut += mine_too ? kOne + (t.at & ((1ull << 40) - 1)) : 0;
        }
        in_cut = wave_total(in_cut);
      }
      m += (double)in_cut * kUnit * edges[cut];
    }
    if (lane == 0) masses[unit] = m;
  }
  __syncthreads();
  double mine = 0.0;
  if (tid < k.segments)
    for (uint32_t i = 0; i < ways; ++i) mine += masses[tid * ways + i];
  const double incl = group_scan(mine, side);
  __syncthreads();
  if (tid == kWide - 1) side[0] = incl;
  if (tid == 0) chosen = 0;
  __syncthreads();
  // (with 1 the last one, whatever rounding does to sums of sums)
  const float u = a.d_u[row];
  const double goal = u < 1.f ? (u > 0.f ? (double)u * side[0] : 0.0) : u >= 1.f ? __builtin_inf() : 0.0;
  // the first segment whose sum passes it; the last with anything if none does
  const uint64_t passes = __ballot(incl > goal && mine > 0.0), has = __ballot(mine > 0.0);
  if (lane == 0 && has)
    atomicMax(&chosen, passes ? 0x80000000u | (kWide - 1 - (64 * wave + __builtin_ctzll(passes)))
                              : 64 * wave + 64 - __builtin_clzll(has));
  __syncthreads();
  const uint32_t seg = chosen & 0x80000000u ? kWide - 1 - (chosen & 0x7FFFFFFFu) : chosen - 1;
  if (tid == seg) side[1] = incl - mine;
  __syncthreads();
  const double before = side[1];
  // Its tokens again: a wave takes a run of them, 64 at a time, and sums their
  // weights; the one that passes the goal lays its weights out in LDS, each lane
  // a run of its own, for the order within.
  const uint32_t first = seg * k.segment + wave * (64 * ROUNDS);
  const Places places(r16, edge);
  float x[ROUNDS];
#pragma unroll
  for (uint32_t j = 0; j < ROUNDS; ++j)   // all on their way at once
    x[j] = value_at(l, min(max(first + 64 * j + lane, head), head + a.vocab - 1) - head);
  double weight[ROUNDS];
  double own = 0.0;
  const auto weigh = [&](auto near_) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t j = 0; j < ROUNDS; ++j) {
      const uint32_t v = first + 64 * j + lane;
      uint32_t excess;
      const uint32_t bin = places.bin_of<decltype(near_)::value>(x[j], excess);
      const bool kept = v >= head && v < head + a.vocab && (bin < cut || (bin == cut && key_of(x[j], v - head) >= tau));
      weight[j] = kept ? (double)(kOne + excess) * kUnit * edges[bin] : 0.0;   // as the bins hold it
      own += weight[j];
    }
  };
  if (places.near_)
    weigh(std::true_type{});
  else
    weigh(std::false_type{});
  for (uint32_t o = 32; o; o >>= 1) own += __shfl_xor(own, o);
  if (lane == 0) masses[wave] = own;   // (what it held has been read)
  __syncthreads();
  // the first wave whose sum passes; the last with anything if none does
  double sum = before;
  uint32_t chosen_wave = 0;
  bool passed = false;
  double each[kWide / 64];
#pragma unroll
  for (uint32_t w2 = 0; w2 < kWide / 64; ++w2) each[w2] = masses[w2];
#pragma unroll
  for (uint32_t w2 = 0; w2 < kWide / 64; ++w2) {
    if (passed) continue;
    if (each[w2] > 0.0) {
      chosen_wave = w2;
      passed = sum + each[w2] > goal;
    }
    if (!passed) sum += each[w2];
  }
  if (wave != chosen_wave) return;
  if (!passed) sum = -1.0;   // its last one, whatever the sums say
  double *const laid = reinterpret_cast<double *>(list);   // nobody else's by now
#pragma unroll
  for (uint32_t j = 0; j < ROUNDS; ++j) laid[64 * j + lane] = weight[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  own = 0.0;
  uint32_t last = 0;   // 1 + this lane's last kept one
  for (uint32_t j = 0; j < ROUNDS; ++j) {
    const double m = laid[lane * ROUNDS + j];
    own += m;
    if (m > 0.0) last = j + 1;
  }
  const double upto_lane = sum + wave_scan(own);
  const uint64_t hits = __ballot(passed && own > 0.0 && upto_lane > goal), any = __ballot(own > 0.0);
  const int at = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(any);
  if ((int)lane == at) {
    uint32_t i = last - 1;
    if (hits) {
      double upto = upto_lane - own;
      for (uint32_t j = 0; j < ROUNDS; ++j) {
        const double m = laid[lane * ROUNDS + j];
        upto += m;
        if (m > 0.0 && (upto > goal || j + 1 == last)) {
          i = j;
          break;
        }
      }
    }
    a.d_token[row] = (int32_t)(first + lane * ROUNDS + i - head);
  }
}

// ---- the kept tokens' probabilities
template <typename T, typename O, uint32_t NT, uint32_t NV>
__global__ __launch_bounds__(NT) void k_probs(SampleKernelArgs k) {
  constexpr uint32_t E = kPiece<T>, S = NT * NV * E;
  const enc_sample_args &a = k.a;
  const uint32_t tid = threadIdx.x, r = blockIdx.x / k.segments, seg = blockIdx.x - r * k.segments;
  __shared__ double edges[kBins];
  const SampleRow &w = k.rows[r];
  const T *l = static_cast<const T *>(a.d_logits) + (uint64_t)(k.row0 + r) * a.logits_row;
  O *out = static_cast<O *>(a.d_probs) + (uint64_t)(k.row0 + r) * a.probs_row;
  const uint32_t head = head_of(l), cut = w.cut_bin;
  uint4 piece[NV];
#pragma unroll
  for (uint32_t j = 0; j < NV; ++j) piece[j] = load_piece(l, head, a.vocab, seg * S + (j * NT + tid) * E);
  const u64 tau = w.tau;
  const bool empty = w.state == kSampleEmpty;
  const double inv = empty ? 0.0 : 1.0 / w.z;
  fill_edges(edges);
  __syncthreads();
  const Places places(w.r16, w.edge);
  // whole pieces of the output where its rows lie as the logits' do
  const bool whole = head_of(out) % E == head && sizeof(O) * E <= 16;
  const auto write = [&](auto near_) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t j = 0; j < NV; ++j) {
      const uint32_t at = seg * S + (j * NT + tid) * E;
      float x[E];
      O p[E];
      values_of<T>(piece[j], x);
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        uint32_t excess;
        const uint32_t bin = places.bin_of<decltype(near_)::value>(x[e], excess);
        float v = 0.f;
        if (!empty && (bin < cut || (bin == cut && key_of(x[e], at + e - head) >= tau)))
          v = (float)((1.0 + (double)excess * kUnit) * edges[bin] * inv);
        p[e] = (O)v;
      }
      typedef O Run __attribute__((ext_vector_type(E)));
      if (whole && at >= head && at + E <= head + a.vocab) {
        Run run;
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) run[e] = p[e];
        *reinterpret_cast<Run *>(out + ((int64_t)at - head)) = run;
      } else {
#pragma unroll
        for (uint32_t e = 0; e < E; ++e)
          if (at + e >= head && at + e < head + a.vocab) out[at + e - head] = p[e];
      }
    }
  };
  if (places.near_)
    write(std::true_type{});
  else
    write(std::false_type{});
}

template <typename T, typename O>
void launch_probs(const SampleKernelArgs &k, uint32_t rows, hipStream_t s) {
  constexpr uint32_t E = kPiece<T>;
  const dim3 grid(rows * k.segments);
  if (k.segment == 4096)
    hipLaunchKernelGGL((k_probs<T, O, 256, 16 / E>), grid, dim3(256), 0, s, k);
  else
    hipLaunchKernelGGL((k_probs<T, O, 512, 32 / E>), grid, dim3(512), 0, s, k);
}

template <typename T>
void launch_rows(const SampleKernelArgs &k, uint32_t rows, hipStream_t s) {
  constexpr uint32_t E = kPiece<T>;
  const dim3 grid(rows * k.segments);
  const bool cuts = k.a.d_top_k || k.a.d_top_p || k.a.d_min_p;
  if (k.segment == 4096)
    hipLaunchKernelGGL((k_scan<T, 256, 16 / E>), grid, dim3(256), 0, s, k);
  else
    hipLaunchKernelGGL((k_scan<T, 512, 32 / E>), grid, dim3(512), 0, s, k);
  hipLaunchKernelGGL(k_plan, dim3(rows), dim3(kWide), 0, s, k);
  if (cuts) {
    if (k.segment == 4096)
      hipLaunchKernelGGL((k_collect<T, 256, 16 / E>), grid, dim3(256), 0, s, k);
    else
      hipLaunchKernelGGL((k_collect<T, 512, 32 / E>), grid, dim3(512), 0, s, k);
  }
  if (k.segment == 4096)
    hipLaunchKernelGGL((k_resolve<T, 4>), dim3(rows), dim3(kWide), 0, s, k);
  else
    hipLaunchKernelGGL((k_resolve<T, 16>), dim3(rows), dim3(kWide), 0, s, k);
  if (k.a.d_probs) {
    if (k.a.probs_dtype == 1)
      launch_probs<T, __bf16>(k, rows, s);
    else if (k.a.probs_dtype == 2)
      launch_probs<T, _Float16>(k, rows, s);
    else
      launch_probs<T, float>(k, rows, s);
  }
}

}  // namespace

// Segments of 16384 values where that leaves every compute unit one, of 4096
// below, where a row's latency counts (the list of segments ends at kSampleSegments). Rows go 1024 at a time through the
// workspace, fewer where they are so long that it would pass some 300 MB.
SamplePlan plan_sample(uint32_t rows, uint32_t vocab) {
  SamplePlan p;
  p.rows = std::min(rows, 1024u);
  const uint64_t large = (vocab + 7ull + 16383) / 16384;
  p.rows = (uint32_t)std::min<uint64_t>(p.rows, 32768 / large);
  p.segment = p.rows * large >= 256 || (vocab + 7ull + 4095) / 4096 > kSampleSegments ? 16384 : 4096;
  p.segments = (uint32_t)((vocab + 7ull + p.segment - 1) / p.segment);
  const uint64_t n = (uint64_t)p.rows * p.segments;
  p.bins = align_up(8ull * kSampleBins * n, 256);
  p.segs = align_up(sizeof(SampleSegment) * n, 256);
  p.sums = align_up(8ull * kSampleBins * p.rows, 256);
  p.row_bytes = align_up(sizeof(SampleRow) * p.rows, 256);
  p.list = align_up(sizeof(SampleToken) * (uint64_t)kSampleList * p.rows, 256);
  return p;
}

// The plan grows with the rows but where it goes over to longer segments.
uint64_t sample_bytes(uint32_t rows, uint32_t vocab) {
  const uint32_t large = (uint32_t)((vocab + 7ull + 16383) / 16384), few = std::min(rows, 255 / large);
  return std::max(plan_sample(rows, vocab).total(), few ? plan_sample(few, vocab).total() : 0);
}

hipError_t launch_sample(SampleKernelArgs k, const SamplePlan &p, hipStream_t s) {
  for (uint64_t row0 = 0; row0 < k.a.rows; row0 += p.rows) {
    k.row0 = (uint32_t)row0;
    const uint32_t rows = std::min(p.rows, k.a.rows - k.row0);
    switch (k.a.dtype) {
      case 1: launch_rows<__bf16>(k, rows, s); break;
      case 2: launch_rows<_Float16>(k, rows, s); break;
      default: launch_rows<float>(k, rows, s); break;
    }
  }
  return hipGetLastError();
}

}  // namespace enc
