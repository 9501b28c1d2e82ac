// step_common.h -- definitions shared by the kernels of one decoding step
// (qk_rope, block_norm, tree_attention, prefix_attention,
// sample, verify_tree, cache_pages) and their host side.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "enc.h"
#include "enc_common.h"

namespace enc {

// Quotients by a divisor known on the host, for n < 2^31: with
// l = ceil(log2 d) and m = ceil(2^(32+l) / d) - 2^32, the high half of m n,
// plus n, shifted right by l, is floor(n / d) (division by invariant
// integers using multiplication; the sum stays below 2^32 because n < 2^31).
struct FastDiv {
  uint32_t d, m, l;
  static FastDiv of(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.l = 0;
    while ((1ull << f.l) < d) ++f.l;
    f.m = (uint32_t)((((1ull << f.l) - d) << 32) / d + 1);
    if ((1ull << f.l) == d) f.m = 0;
    return f;
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two fp32 values rounded to nearest even, packed low half first.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__bf16>(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
template <> __device__ __forceinline__ uint32_t pack2<_Float16>(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}
template <typename T> __device__ __forceinline__ float half_of(uint32_t v, int hi);
template <> __device__ __forceinline__ float half_of<__bf16>(uint32_t v, int hi) {
  return __uint_as_float(hi ? v & 0xFFFF0000u : v << 16);
}
template <> __device__ __forceinline__ float half_of<_Float16>(uint32_t v, int hi) {
  return (float)__builtin_bit_cast(f16x2, v)[hi];
}

struct QkKernelArgs {
  enc_qk_args a;
  uint32_t heads;      // that a token has: q, k and, if given, v
  uint32_t vec;        // angles in aligned runs of 4
  FastDiv blocks;      // workgroups to a token
  uint32_t token0;     // this launch's first
};
hipError_t launch_qk_norm_rope(const QkKernelArgs &k, hipStream_t s);

struct BlockNormKernelArgs {
  enc_block_norm_args a;
  FastDiv gate;        // tokens to a row of gates
  uint32_t vec;        // all rows and weights 16-byte aligned, width a multiple of 8
  uint32_t token0;     // this launch's first
};
hipError_t launch_block_norm(const BlockNormKernelArgs &k, hipStream_t s);

struct TreeAttnArgs {
  enc_tree_attention_args a;
  FastDiv page, group;       // page_size; q_heads / kv_heads
  uint32_t rows;             // nodes * group: query rows that share a KV head
  uint32_t row_tiles;        // tiles of rows, each one workgroup's
  uint32_t parts;            // equal parts the call's keys are cut into
  uint32_t grid_parts;       // and the most there are, with short last ones
  uint32_t least;            // units in the smallest part
  uint32_t mask_words;       // 32-bit mask words per node
  float *part;               // [grid_parts, kv_heads, rows, head_dim] unnormalised sums
  float *part_ml;            // [grid_parts, kv_heads, rows, 2] running maximum and sum
  uint2 *shares;             // [batch] first part and number of parts; NULL: never more than one
  uint32_t raw;              // maxima are of q.k times the scale's sign, not yet scaled
  float unit;                // powers of two to a unit of a maximum
  float slack;               // how far a strip may exceed it before it moves
};
struct TreeAttnPlan {
  uint32_t wide;             // rows on different waves, keys through LDS
  uint32_t units, waves;     // 16-row units a wave holds; waves of a workgroup
  uint32_t ways, unit;       // waves that take different keys; keys in a unit of work
  uint32_t row_tiles, parts, grid_parts, least;
  uint64_t part_bytes, ml_bytes, share_bytes;
};
TreeAttnPlan plan_tree_attention(const enc_tree_attention_args &a);
hipError_t launch_tree_attention(TreeAttnArgs k, const TreeAttnPlan &p, hipStream_t s);

struct VerifyKernelArgs {
  enc_verify_args a;
  uint32_t groups;           // workgroups per sequence
  uint32_t segment;          // elements a wave sums at a time (multiple of 256)
  uint32_t spins;            // polls before a workgroup goes on alone
  unsigned long long *totals;// [batch, 2, groups * 16] sums of two rounds' segments
  uint32_t *done;            // [batch] workgroups that are through
};
struct VerifyPlan {
  uint32_t groups, segment;
  uint64_t totals_bytes, done_bytes;
};
VerifyPlan plan_verify_tree(uint32_t batch, uint32_t vocab);
hipError_t launch_verify_tree(const VerifyKernelArgs &k, hipStream_t s);

// A piece's work: a tile of query rows over a range of keys.
struct PrefixItem {
  uint32_t b, row0, rows;    // first batch entry, first row of its rows, and how many
  uint32_t first, ctx, tree; // first cached token, how many, and nodes behind them
  uint32_t lo, hi;           // strips of 32 keys
  uint32_t turn;             // heads are taken from this one on
  uint32_t seq;              // row of the table
};
struct PrefixAttnArgs {
  enc_tree_attention_args a;
  const int32_t *starts, *shared;
  FastDiv page, group, nodes;   // page_size; q_heads / kv_heads; nodes
  uint32_t groups;
  uint32_t tile, own_tile, own_tiles;   // rows of a tile; tiles of a sequence's rows
  uint32_t slots, own_slots, least;     // pieces aimed at; strips in the smallest
  uint32_t mask_words;
  float unit;                // powers of two to a unit of a maximum
  float slack, half_slack;   // how far a strip may exceed it; half of that
  uint64_t own_rows;         // of the pieces of own tokens, the first
  float *part, *part_ml;     // [pieces, kv_heads, tile, head_dim], [.., 2] sums; maxima and weights' sums
  PrefixItem *items;
  uint32_t *first, *group_of;   // [batch] tokens shared; group, or ~0
  uint2 *own_parts;          // [batch] first piece and how many
  uint32_t *ends, *common;   // [groups + 1] batch entries; [groups] tokens shared
  uint2 *group_parts;        // [groups] first piece and how many
  uint32_t *counts;          // pieces of shared tokens; of all
};
struct PrefixAttnPlan {
  uint32_t tile, own_tile, own_tiles, slots, own_slots, least, most_shared, most_own, items;
  uint64_t part_bytes, ml_bytes, item_bytes, batch_bytes, group_bytes;
  uint64_t total() const { return part_bytes + ml_bytes + item_bytes + 4 * batch_bytes + 4 * group_bytes + 256; }
};
PrefixAttnPlan plan_prefix_attention(const enc_tree_attention_args &a, uint32_t groups);
uint64_t prefix_attention_bytes(const enc_tree_attention_args &a, uint32_t groups);   // for it and all smaller calls
hipError_t launch_prefix_attention(PrefixAttnArgs k, const PrefixAttnPlan &p, hipStream_t s);
hipError_t launch_cache_shared(const enc_cache &c, const int32_t *seqs, uint32_t batch, const int32_t *starts,
                               uint32_t groups, int32_t *shared, hipStream_t s);

// What the passes over a row of logits hand on (see sample.hip).
constexpr uint32_t kSampleBins = 768, kSampleList = 4096, kSampleSegments = 1024;
enum : uint32_t { kSampleEmpty, kSampleFirst, kSampleWhole, kSampleListed, kSampleRead };
struct SampleSegment {
  unsigned long long top;    // greatest key, 0: none
  double edge;               // its bin's place
  uint32_t bins;             // written bins, from there down
  uint32_t n, first;         // tokens gathered from it, and their place in the list
  uint32_t reserved;
};
struct SampleRow {
  double edge, r16;          // place of the first bin; 16 / temperature
  double t_min, top_p, z;    // min-p's least place; kept weights' sum
  unsigned long long top, tau;  // greatest key; the least that is kept of the cut's bin (0: all)
  uint32_t state;            // kSample...
  uint32_t bk, lo, hi, bm;   // bins in which top-k, top-p (from, to) and min-p cut, or ~0
  uint32_t kb, rank;         // last bin that top-k reaches, and how many tokens of it
  uint32_t bk_n, lo_n;       // tokens of bin bk; of bin lo, if that is hi
  uint32_t cut_bin, n;       // the cut's bin; tokens to gather
};
struct SampleToken {
  unsigned long long key, at;   // at: bin in the upper 24 bits, weight less 1 in units of 2^-32
};
struct SampleKernelArgs {
  enc_sample_args a;
  uint32_t row0, segment, segments;
  unsigned long long *bins;  // [rows, segments, kSampleBins] count in the upper 15 bits, sum below
  SampleSegment *segs;       // [rows, segments]
  double *sums;              // [rows, kSampleBins] cumulative weights
  SampleRow *rows;           // [rows]
  SampleToken *list;         // [rows, kSampleList]
};
struct SamplePlan {
  uint32_t rows;             // at a time
  uint32_t segment, segments;
  uint64_t bins, segs, sums, row_bytes, list;   // bytes of the workspace's parts
  uint64_t total() const { return bins + segs + sums + row_bytes + list; }
};
SamplePlan plan_sample(uint32_t rows, uint32_t vocab);
uint64_t sample_bytes(uint32_t rows, uint32_t vocab);   // for it and all calls of fewer rows
hipError_t launch_sample(SampleKernelArgs k, const SamplePlan &p, hipStream_t s);

struct CommitArgs {
  enc_cache c;
  FastDiv page;
  const int32_t *seqs, *path, *count;
  const uint8_t *draft;
  uint64_t draft_plane, draft_seq;
  uint32_t batch, nodes;
  int32_t *status;
  int32_t *info;             // [batch, 4] length before, rows, page copied from (or -1), page copied to
  int32_t *first;            // [batch] rank of the sequence's first new page
  int32_t *pick;             // [pages the call may need] free pages by rank
  int32_t *to;               // [batch, nodes] cache row of each accepted row, -1 past them
};
hipError_t launch_cache_commit(const CommitArgs &k, hipStream_t s);
hipError_t launch_cache_fork(const enc_cache &c, const int32_t *src, const int32_t *dst, uint32_t pairs,
                             hipStream_t s);
hipError_t launch_cache_truncate(const enc_cache &c, const int32_t *seqs, const int32_t *lens,
                                 uint32_t count, hipStream_t s);

enc_status after_launch(hipError_t e, hipStream_t s, const char *what);

}  // namespace enc
