// step_api.cpp -- host side of the decoding-step entry points (head norms with
// rotation, tree attention, verification, cache pages): every argument that
// the host can see is checked before anything is launched.
#include "enc.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdlib>

#include "enc_common.h"
#include "step_common.h"

using namespace enc;

namespace {

bool aligned(const void *p, uint64_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uint32_t value_bytes(uint32_t dtype) { return dtype == 3 ? 4u : 2u; }

enc_status invalid(const char *what) { return set_error(ENC_ERR_INVALID_ARG, "%s", what); }
enc_status unsupported(const char *what) { return set_error(ENC_ERR_UNSUPPORTED, "%s", what); }

// An array of [.., .., head_dim] values: 16-byte aligned base and rows.
bool rows_ok(const void *p, uint32_t dtype, uint64_t s0, uint64_t s1, uint64_t s2 = 0) {
  const uint64_t per = 16 / value_bytes(dtype);
  return p && aligned(p, 16) && s0 % per == 0 && s1 % per == 0 && s2 % per == 0;
}

enc_status check_attention(const enc_tree_attention_args *a) {
  if (!a) return invalid("args is NULL");
  if (a->reserved != 0) return invalid("reserved is not 0");
  if (a->dtype != 1 && a->dtype != 2) return unsupported("attention takes BF16 and FP16");
  if (!a->nodes || !a->q_heads || !a->kv_heads || !a->head_dim || !a->page_size || !a->n_pages || !a->max_pages ||
      !a->max_seqs)
    return invalid("a size is 0");
  if (a->nodes > ENC_TREE_MAX_NODES) return unsupported("more nodes than ENC_TREE_MAX_NODES");
  if (a->head_dim % 8 || a->head_dim > 256) return unsupported("head_dim must be a multiple of 8 up to 256");
  if (a->q_heads % a->kv_heads) return set_error(ENC_ERR_SHAPE, "%u query heads over %u KV heads", a->q_heads, a->kv_heads);
  if (a->page_size > 65536) return unsupported("page_size above 65536");
  if ((uint64_t)a->max_pages * a->page_size > 0x7FFFFFFFull) return unsupported("max_pages * page_size above 2^31 - 1");
  const uint64_t rows = (uint64_t)a->nodes * (a->q_heads / a->kv_heads);
  if (rows > 65536) return unsupported("more than 65536 query rows share a KV head");
  // a grid holds fewer than 2^32 threads
  if ((uint64_t)a->batch * a->kv_heads * rows > (1ull << 25) || (uint64_t)a->batch * a->kv_heads > (1ull << 23))
    return unsupported("batch * nodes * q_heads above 2^25, or batch * kv_heads above 2^23");
  if ((uint64_t)a->n_pages * a->page_size > 0x7FFFFFFFull) return unsupported("n_pages * page_size above 2^31 - 1");
  if (((uint64_t)a->max_pages * a->page_size / 32 + 16) * a->batch > 0xFFFFFFFFull)
    return unsupported("batch * max_pages * page_size above 2^37");
  return ENC_OK;
}

enc_status check_attention_arrays(const enc_tree_attention_args *a) {
  if (!std::isfinite(a->scale)) return invalid("scale is not finite");
  if (!rows_ok(a->d_q, a->dtype, a->q_batch, a->q_node, a->q_head) ||
      !rows_ok(a->d_out, a->dtype, a->out_batch, a->out_node, a->out_head))
    return invalid("q or out: NULL, or a base or row that is not 16-byte aligned");
  if (!rows_ok(a->d_k_new, a->dtype, a->k_new_batch, a->k_new_node, a->k_new_head) ||
      !rows_ok(a->d_v_new, a->dtype, a->v_new_batch, a->v_new_node, a->v_new_head))
    return invalid("k_new or v_new: NULL, or a base or row that is not 16-byte aligned");
  if (!rows_ok(a->d_k_cache, a->dtype, a->cache_page, a->cache_token, a->cache_head) ||
      !rows_ok(a->d_v_cache, a->dtype, 0, 0))
    return invalid("cache: NULL, or a base or row that is not 16-byte aligned");
  if (!a->d_table || !a->d_lens || !aligned(a->d_table, 4) || !aligned(a->d_lens, 4) || !aligned(a->d_seqs, 4) ||
      !aligned(a->d_nodes, 4) || !aligned(a->d_mask, 8) || !aligned(a->d_lse, 4))
    return invalid("table or lens NULL, or a misaligned array");
  if (!a->d_seqs && a->batch > a->max_seqs) return invalid("without seqs, batch must not exceed max_seqs");
  // row offsets are kept in 16-byte units of 32 bits: each layer's cache below 64 GiB
  const uint64_t reach = (uint64_t)(a->n_pages - 1) * (a->cache_page / 8) + (uint64_t)(a->page_size - 1) * (a->cache_token / 8);
  if (a->cache_page >> 35 || a->cache_token >> 35 || reach >> 32) return unsupported("a cache above 64 GiB");
  if ((a->nodes - 1ull) * (a->k_new_node / 8) >> 31 || (a->nodes - 1ull) * (a->v_new_node / 8) >> 31 ||
      a->k_new_node >> 35 || a->v_new_node >> 35)
    return unsupported("k_new or v_new strides above 32 GiB");
  return ENC_OK;
}

enc_status check_cache(const enc_cache *c) {
  if (!c) return invalid("cache is NULL");
  if (!c->d_data || !c->d_table || !c->d_lens || !c->d_refs) return invalid("a pointer of the cache is NULL");
  if (!c->n_planes || !c->n_pages || !c->page_size || !c->row_bytes || !c->max_seqs || !c->max_pages)
    return invalid("a size of the cache is 0");
  if (!aligned(c->d_data, 16) || c->plane_stride % 16 || c->row_bytes % 16)
    return invalid("cache data, plane_stride and row_bytes must be multiples of 16");
  if (!aligned(c->d_table, 4) || !aligned(c->d_lens, 4) || !aligned(c->d_refs, 4))
    return invalid("a cache array is misaligned");
  if (c->n_planes > 65535 || c->page_size > 65536 || c->n_pages > 0x7FFFFFFFu || c->max_seqs > 0x7FFFFFFFu)
    return unsupported("n_planes above 65535, page_size above 65536, or 2^31 pages or sequences");
  if ((uint64_t)c->max_pages * c->page_size > 0x7FFFFFFFull) return unsupported("max_pages * page_size above 2^31 - 1");
  // a row is copied by steps of up to 4096 bytes, counted in 32 bits
  if (c->row_bytes > (1u << 31)) return unsupported("row_bytes above 2^31");
  const uint64_t used = (uint64_t)c->n_pages * c->page_size;
  if (used > 0x7FFFFFFFull) return unsupported("n_pages * page_size above 2^31 - 1");
  if (used > (1ull << 40) / c->row_bytes) return unsupported("a plane above 2^40 bytes");
  if (c->n_planes > 1 && c->plane_stride < used * c->row_bytes) return invalid("plane_stride below a plane's bytes");
  return ENC_OK;
}

enc_status check_prefix(const enc_prefix_attention_args *a) {
  if (!a) return invalid("args is NULL");
  if (a->reserved != 0) return invalid("reserved is not 0");
  const enc_status st = check_attention(&a->t);
  if (st != ENC_OK) return st;
  if (a->groups > (1u << 20)) return unsupported("more than 2^20 groups");
  if (a->t.batch) {   // a grid holds fewer than 2^32 threads
    const PrefixAttnPlan p = plan_prefix_attention(a->t, a->groups);
    if ((uint64_t)p.items * a->t.kv_heads >= (1u << 23)) return unsupported("more than 2^23 pieces");
  }
  return ENC_OK;
}

struct CommitLayout {
  uint64_t info, first, pick, to, total;
};
CommitLayout commit_layout(const enc_cache *c, uint32_t batch, uint32_t nodes) {
  CommitLayout l;
  l.info = 0;
  l.first = align_up(16ull * batch, 256);
  l.pick = l.first + align_up(4ull * batch, 256);
  // a sequence's rows reach at most this many pages
  const uint64_t reach = (nodes + c->page_size - 1) / c->page_size + 1;
  l.to = l.pick + align_up(4ull * batch * reach, 256);
  l.total = l.to + align_up(4ull * batch * nodes, 256);
  return l;
}

}  // namespace

extern "C" {

enc_status enc_qk_norm_rope(const enc_qk_args *a, void *stream) {
  set_error(ENC_OK, "%s", "");
  if (!a) return invalid("args is NULL");
  if (a->reserved != 0 || (a->flags & ~(ENC_ROPE_ADJACENT | ENC_QK_NO_NORM))) return invalid("unknown flags");
  if (a->in_dtype - 1u > 2u || a->out_dtype - 1u > 2u || a->w_dtype - 1u > 2u) return unsupported("unknown dtype");
  if (!a->q_heads || !a->kv_heads || !a->head_dim) return invalid("a size is 0");
  if (a->head_dim % 8 || a->head_dim > 512) return unsupported("head_dim must be a multiple of 8 up to 512");
  if (a->rot_dim % 2 || a->rot_dim > a->head_dim) return invalid("rot_dim must be even and at most head_dim");
  if (!(a->flags & ENC_QK_NO_NORM) && !(a->eps >= 0.f && std::isfinite(a->eps))) return invalid("eps must be finite and >= 0");
  if (a->tokens == 0) return ENC_OK;
  if (!rows_ok(a->d_q, a->in_dtype, a->q_token, a->q_head) || !rows_ok(a->d_k, a->in_dtype, a->k_token, a->k_head) ||
      !rows_ok(a->d_q_out, a->out_dtype, a->q_out_token, a->q_out_head) ||
      !rows_ok(a->d_k_out, a->out_dtype, a->k_out_token, a->k_out_head))
    return invalid("q or k: NULL, or a base or row that is not 16-byte aligned");
  if (a->d_v && (!rows_ok(a->d_v, a->in_dtype, a->v_token, a->v_head) ||
                 !rows_ok(a->d_v_out, a->out_dtype, a->v_out_token, a->v_out_head)))
    return invalid("v: no output, or a base or row that is not 16-byte aligned");
  if ((a->d_q_weight && !aligned(a->d_q_weight, 16)) || (a->d_k_weight && !aligned(a->d_k_weight, 16)))
    return invalid("a weight is not 16-byte aligned");
  if (a->rot_dim && (!a->d_positions || !a->d_table || !a->max_pos || !aligned(a->d_positions, 4) || !aligned(a->d_table, 4)))
    return invalid("rotation needs positions and a table");
  if (a->max_pos > 0x7FFFFFFFu) return unsupported("max_pos above 2^31 - 1");
  const uint64_t heads = (uint64_t)a->q_heads + a->kv_heads * (a->d_v ? 2ull : 1ull);
  if (heads > 65536 || heads * a->tokens > 0x7FFFFFFFull) return unsupported("more than 65536 heads, or tokens * heads above 2^31 - 1");
  QkKernelArgs k;
  k.a = *a;
  k.heads = (uint32_t)heads;
  k.vec = a->rot_dim % (a->flags & ENC_ROPE_ADJACENT ? 8 : 16) == 0 && aligned(a->d_table, 16);
  k.blocks = FastDiv::of(1);
  return after_launch(launch_qk_norm_rope(k, (hipStream_t)stream), (hipStream_t)stream, "enc_qk_norm_rope");
}

enc_status enc_block_norm(const enc_block_norm_args *a, void *stream) {
  set_error(ENC_OK, "%s", "");
  if (!a) return invalid("args is NULL");
  if (a->flags & ~(ENC_BLOCK_POST_NORM | ENC_BLOCK_UNIT_OFFSET)) return invalid("unknown flags");
  if (!a->width) return invalid("width is 0");
  if (a->width > 32768) return unsupported("width above 32768");
  if (!(a->eps >= 0.f && std::isfinite(a->eps))) return invalid("eps must be finite and >= 0");
  if (!std::isfinite(a->h_scale) || !std::isfinite(a->y_scale)) return invalid("h_scale and y_scale must be finite");
  if (a->tokens == 0) return ENC_OK;
  if (a->tokens > 0x7FFFFFFFu) return unsupported("tokens above 2^31 - 1");
  if (!a->d_h || (!a->d_h_out && !a->d_out)) return invalid("h is NULL, or no output is asked for");
  if (!a->d_y && (a->d_gate || (a->flags & ENC_BLOCK_POST_NORM))) return invalid("a gate or a norm of y without y");
  if (a->d_w_post && !(a->flags & ENC_BLOCK_POST_NORM)) return invalid("w_post without ENC_BLOCK_POST_NORM");
  if (a->d_w_pre && !a->d_out) return invalid("w_pre without out");
  if (a->d_gate && !a->gate_every) return invalid("gate_every is 0");
  const struct {
    const void *p;
    uint32_t dtype;
    uint64_t stride;
    bool out;
  } arrays[] = {{a->d_y, a->y_dtype, a->y_token, false},        {a->d_h, a->h_dtype, a->h_token, false},
                {a->d_gate, a->g_dtype, a->gate_row, false},    {a->d_w_post, a->w_dtype, 0, false},
                {a->d_w_pre, a->w_dtype, 0, false},             {a->d_h_out, a->h_dtype, a->h_out_token, true},
                {a->d_out, a->out_dtype, a->out_token, true}};
  bool vec = a->width % 8 == 0;
  for (const auto &x : arrays) {
    if (!x.p) continue;
    if (x.dtype - 1u > 2u) return unsupported("unknown dtype");
    if (!aligned(x.p, value_bytes(x.dtype))) return invalid("a misaligned array");
    if (x.stride >> 40) return unsupported("a stride of 2^40 or more");
    if (x.out && a->tokens > 1 && x.stride < a->width) return invalid("rows of an output overlap");
    vec = vec && aligned(x.p, 16) && x.stride % (16 / value_bytes(x.dtype)) == 0;
  }
  BlockNormKernelArgs k;
  k.a = *a;
  k.gate = FastDiv::of(a->d_gate ? a->gate_every < 0x80000000u ? a->gate_every : 0x7FFFFFFFu : 1);
  k.vec = vec;
  k.token0 = 0;
  return after_launch(launch_block_norm(k, (hipStream_t)stream), (hipStream_t)stream, "enc_block_norm");
}

uint64_t enc_tree_attention_workspace_bytes(const enc_tree_attention_args *a) {
  set_error(ENC_OK, "%s", "");
  if (check_attention(a) != ENC_OK || a->batch == 0) return 0;
  const TreeAttnPlan p = plan_tree_attention(*a);
  return p.part_bytes + p.ml_bytes + p.share_bytes;
}

enc_status enc_tree_attention(const enc_tree_attention_args *a, void *d_ws, uint64_t ws_bytes, void *stream) {
  set_error(ENC_OK, "%s", "");
  const enc_status st = check_attention(a);
  if (st != ENC_OK) return st;
  if (a->batch == 0) return ENC_OK;
  const enc_status ar = check_attention_arrays(a);
  if (ar != ENC_OK) return ar;
  const TreeAttnPlan p = plan_tree_attention(*a);
  const uint64_t need = p.part_bytes + p.ml_bytes + p.share_bytes;
  if (need) {
    if (!d_ws || !aligned(d_ws, 16)) return invalid("workspace is NULL or not 16-byte aligned");
    if (ws_bytes < need)
      return set_error(ENC_ERR_CAPACITY, "workspace of %llu bytes, %llu needed", (unsigned long long)ws_bytes,
                       (unsigned long long)need);
  }
  TreeAttnArgs k;
  k.a = *a;
  k.page = FastDiv::of(a->page_size);
  k.group = FastDiv::of(a->q_heads / a->kv_heads);
  k.rows = a->nodes * (a->q_heads / a->kv_heads);
  k.row_tiles = p.row_tiles;
  k.parts = p.parts;
  k.grid_parts = p.grid_parts;
  k.least = p.least;
  k.mask_words = (a->nodes + 63) / 64 * 2;
  k.part = static_cast<float *>(d_ws);
  k.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(d_ws) + p.part_bytes);
  k.shares = need ? reinterpret_cast<uint2 *>(static_cast<uint8_t *>(d_ws) + p.part_bytes + p.ml_bytes) : nullptr;
  return after_launch(launch_tree_attention(k, p, (hipStream_t)stream), (hipStream_t)stream, "enc_tree_attention");
}

uint64_t enc_prefix_attention_workspace_bytes(const enc_prefix_attention_args *a) {
  set_error(ENC_OK, "%s", "");
  if (check_prefix(a) != ENC_OK || a->t.batch == 0) return 0;
  return prefix_attention_bytes(a->t, a->groups);
}

enc_status enc_prefix_attention(const enc_prefix_attention_args *a, void *d_ws, uint64_t ws_bytes, void *stream) {
  set_error(ENC_OK, "%s", "");
  enc_status st = check_prefix(a);
  if (st != ENC_OK) return st;
  const enc_tree_attention_args &t = a->t;
  if (t.batch == 0) return ENC_OK;
  if ((st = check_attention_arrays(&t)) != ENC_OK) return st;
  if (a->groups && (!a->d_starts || !a->d_shared || !aligned(a->d_starts, 4) || !aligned(a->d_shared, 4)))
    return invalid("starts or shared NULL or misaligned");
  const PrefixAttnPlan p = plan_prefix_attention(t, a->groups);
  if (!d_ws || !aligned(d_ws, 16)) return invalid("workspace is NULL or not 16-byte aligned");
  if (ws_bytes < p.total())
    return set_error(ENC_ERR_CAPACITY, "workspace of %llu bytes, %llu needed", (unsigned long long)ws_bytes,
                     (unsigned long long)p.total());
  PrefixAttnArgs k;
  k.a = t;
  k.starts = a->d_starts;
  k.shared = a->d_shared;
  k.page = FastDiv::of(t.page_size);
  k.group = FastDiv::of(t.q_heads / t.kv_heads);
  k.nodes = FastDiv::of(t.nodes);
  k.groups = a->groups;
  k.tile = p.tile;
  k.own_tile = p.own_tile;
  k.own_tiles = p.own_tiles;
  k.slots = p.slots;
  k.least = p.least;
  k.own_slots = p.own_slots;
  k.mask_words = (t.nodes + 63) / 64 * 2;
  k.own_rows = (uint64_t)p.most_shared * t.kv_heads * p.tile;
  uint8_t *ws = static_cast<uint8_t *>(d_ws);
  k.part = reinterpret_cast<float *>(ws);
  k.part_ml = reinterpret_cast<float *>(ws += p.part_bytes);
  k.items = reinterpret_cast<PrefixItem *>(ws += p.ml_bytes);
  k.first = reinterpret_cast<uint32_t *>(ws += p.item_bytes);
  k.group_of = reinterpret_cast<uint32_t *>(ws += p.batch_bytes);
  k.own_parts = reinterpret_cast<uint2 *>(ws += p.batch_bytes);
  k.ends = reinterpret_cast<uint32_t *>(ws += 2 * p.batch_bytes);
  k.common = reinterpret_cast<uint32_t *>(ws += p.group_bytes);
  k.group_parts = reinterpret_cast<uint2 *>(ws += p.group_bytes);
  k.counts = reinterpret_cast<uint32_t *>(ws += 2 * p.group_bytes);
  return after_launch(launch_prefix_attention(k, p, (hipStream_t)stream), (hipStream_t)stream, "enc_prefix_attention");
}

uint64_t enc_verify_tree_workspace_bytes(uint32_t batch, uint32_t nodes, uint32_t vocab) {
  set_error(ENC_OK, "%s", "");
  if (!batch || !nodes || nodes > ENC_TREE_MAX_NODES || !vocab || vocab > (1u << 22) || batch > (1u << 20)) return 0;
  const VerifyPlan p = plan_verify_tree(batch, vocab);
  return p.totals_bytes + p.done_bytes;
}

enc_status enc_verify_tree(const enc_verify_args *a, void *d_ws, uint64_t ws_bytes, void *stream) {
  set_error(ENC_OK, "%s", "");
  if (!a) return invalid("args is NULL");
  if (a->dtype - 1u > 2u) return unsupported("unknown dtype");
  if (a->batch == 0) return ENC_OK;
  if (!a->nodes || !a->vocab) return invalid("a size is 0");
  if (a->nodes > ENC_TREE_MAX_NODES) return unsupported("more nodes than ENC_TREE_MAX_NODES");
  if (a->vocab > (1u << 22) || a->batch > (1u << 20)) return unsupported("vocab above 2^22 or batch above 2^20");
  const uint32_t vb = value_bytes(a->dtype);
  if (!a->d_parents || !a->d_tokens || !a->d_target || !a->d_u || !a->d_path || !a->d_count || !a->d_token)
    return invalid("a required pointer is NULL");
  if (!aligned(a->d_target, vb) || !aligned(a->d_draft, vb) || !aligned(a->d_parents, 4) || !aligned(a->d_tokens, 4) ||
      !aligned(a->d_u, 4) || !aligned(a->d_nodes, 4) || !aligned(a->d_path, 4) || !aligned(a->d_count, 4) ||
      !aligned(a->d_token, 4))
    return invalid("a misaligned array");
  const VerifyPlan p = plan_verify_tree(a->batch, a->vocab);
  if ((a->batch + 7ull) / 8 * 8 * p.groups > (1u << 21))   // a grid holds fewer than 2^32 threads
    return unsupported("batch * vocab: more than 2^21 workgroups");
  const uint64_t need = p.totals_bytes + p.done_bytes;
  if (!d_ws || !aligned(d_ws, 16)) return invalid("workspace is NULL or not 16-byte aligned");
  if (ws_bytes < need)
    return set_error(ENC_ERR_CAPACITY, "workspace of %llu bytes, %llu needed", (unsigned long long)ws_bytes,
                     (unsigned long long)need);
  VerifyKernelArgs k;
  k.a = *a;
  k.groups = p.groups;
  k.segment = p.segment;
  const char *spins = getenv("ENC_VERIFY_SPINS");
  k.spins = spins && spins[0] ? (uint32_t)strtoul(spins, nullptr, 10) : 1u << 16;
  k.totals = static_cast<unsigned long long *>(d_ws);
  k.done = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(d_ws) + p.totals_bytes);
  return after_launch(launch_verify_tree(k, (hipStream_t)stream), (hipStream_t)stream, "enc_verify_tree");
}

uint64_t enc_sample_workspace_bytes(uint32_t rows, uint32_t vocab) {
  set_error(ENC_OK, "%s", "");
  if (!rows || rows > (1u << 20) || !vocab || vocab > (1u << 22)) return 0;
  return sample_bytes(rows, vocab);
}

enc_status enc_sample(const enc_sample_args *a, void *d_ws, uint64_t ws_bytes, void *stream) {
  set_error(ENC_OK, "%s", "");
  if (!a) return invalid("args is NULL");
  if (a->reserved != 0) return invalid("reserved is not 0");
  if (a->dtype - 1u > 2u || (a->d_probs && a->probs_dtype - 1u > 2u)) return unsupported("unknown dtype");
  if (!a->vocab) return invalid("vocab is 0");
  if (a->vocab > (1u << 22) || a->rows > (1u << 20)) return unsupported("vocab above 2^22 or rows above 2^20");
  if (a->rows == 0) return ENC_OK;
  if (!a->d_logits || (!a->d_token && !a->d_probs)) return invalid("logits is NULL, or no output is asked for");
  if (a->d_token && !a->d_u) return invalid("a token needs u");
  if (!a->rows_per_setting) return invalid("rows_per_setting is 0");
  if (!aligned(a->d_logits, value_bytes(a->dtype)) || (a->d_probs && !aligned(a->d_probs, value_bytes(a->probs_dtype))) ||
      !aligned(a->d_u, 4) || !aligned(a->d_temperature, 4) || !aligned(a->d_top_p, 4) || !aligned(a->d_min_p, 4) ||
      !aligned(a->d_top_k, 4) || !aligned(a->d_token, 4))
    return invalid("a misaligned array");
  if (a->logits_row >> 40 || a->probs_row >> 40) return unsupported("a stride of 2^40 or more");
  if (a->d_probs && a->rows > 1 && a->probs_row < a->vocab) return invalid("rows of probs overlap");
  const SamplePlan p = plan_sample(a->rows, a->vocab);
  const uint64_t need = p.total();
  if (!d_ws || !aligned(d_ws, 16)) return invalid("workspace is NULL or not 16-byte aligned");
  if (ws_bytes < need)
    return set_error(ENC_ERR_CAPACITY, "workspace of %llu bytes, %llu needed", (unsigned long long)ws_bytes,
                     (unsigned long long)need);
  SampleKernelArgs k;
  k.a = *a;
  k.row0 = 0;
  k.segment = p.segment;
  k.segments = p.segments;
  uint8_t *ws = static_cast<uint8_t *>(d_ws);
  k.bins = reinterpret_cast<unsigned long long *>(ws);
  k.segs = reinterpret_cast<SampleSegment *>(ws += p.bins);
  k.sums = reinterpret_cast<double *>(ws += p.segs);
  k.rows = reinterpret_cast<SampleRow *>(ws += p.sums);
  k.list = reinterpret_cast<SampleToken *>(ws += p.row_bytes);
  return after_launch(launch_sample(k, p, (hipStream_t)stream), (hipStream_t)stream, "enc_sample");
}

uint64_t enc_cache_workspace_bytes(const enc_cache *c, uint32_t batch, uint32_t nodes) {
  set_error(ENC_OK, "%s", "");
  if (check_cache(c) != ENC_OK || !batch || batch > (1u << 20) || !nodes || nodes > ENC_TREE_MAX_NODES) return 0;
  return commit_layout(c, batch, nodes).total;
}

enc_status enc_cache_commit(const enc_cache *c, const int32_t *d_seqs, uint32_t batch, const void *d_draft,
                            uint64_t draft_plane, uint64_t draft_seq, const int32_t *d_path, const int32_t *d_count,
                            uint32_t nodes, int32_t *d_status, void *d_ws, uint64_t ws_bytes, void *stream) {
  set_error(ENC_OK, "%s", "");
  const enc_status st = check_cache(c);
  if (st != ENC_OK) return st;
  if (!nodes) return invalid("nodes is 0");
  if (nodes > ENC_TREE_MAX_NODES) return unsupported("more nodes than ENC_TREE_MAX_NODES");
  if (batch > (1u << 20)) return unsupported("batch above 2^20");
  if (!d_status || !aligned(d_status, 4)) return invalid("status is NULL or misaligned");
  if (!batch) return invalid("batch is 0");
  if (!d_seqs || !d_draft || !d_path || !d_count || !aligned(d_seqs, 4) || !aligned(d_path, 4) || !aligned(d_count, 4))
    return invalid("seqs, draft, path or count NULL or misaligned");
  if (!aligned(d_draft, 16) || draft_plane % 16 || draft_seq % 16) return invalid("draft rows must be 16-byte aligned");
  const CommitLayout l = commit_layout(c, batch, nodes);
  if (!d_ws || !aligned(d_ws, 16)) return invalid("workspace is NULL or not 16-byte aligned");
  if (ws_bytes < l.total)
    return set_error(ENC_ERR_CAPACITY, "workspace of %llu bytes, %llu needed", (unsigned long long)ws_bytes,
                     (unsigned long long)l.total);
  CommitArgs k;
  k.c = *c;
  k.page = FastDiv::of(c->page_size);
  k.seqs = d_seqs;
  k.path = d_path;
  k.count = d_count;
  k.draft = static_cast<const uint8_t *>(d_draft);
  k.draft_plane = draft_plane;
  k.draft_seq = draft_seq;
  k.batch = batch;
  k.nodes = nodes;
  k.status = d_status;
  uint8_t *ws = static_cast<uint8_t *>(d_ws);
  k.info = reinterpret_cast<int32_t *>(ws + l.info);
  k.first = reinterpret_cast<int32_t *>(ws + l.first);
  k.pick = reinterpret_cast<int32_t *>(ws + l.pick);
  k.to = reinterpret_cast<int32_t *>(ws + l.to);
  return after_launch(launch_cache_commit(k, (hipStream_t)stream), (hipStream_t)stream, "enc_cache_commit");
}

enc_status enc_cache_fork(const enc_cache *c, const int32_t *d_src, const int32_t *d_dst, uint32_t pairs, void *stream) {
  set_error(ENC_OK, "%s", "");
  const enc_status st = check_cache(c);
  if (st != ENC_OK) return st;
  if (!pairs) return ENC_OK;
  if (pairs > 65535) return unsupported("more than 65535 pairs");
  if (!d_src || !d_dst || !aligned(d_src, 4) || !aligned(d_dst, 4)) return invalid("src or dst NULL or misaligned");
  return after_launch(launch_cache_fork(*c, d_src, d_dst, pairs, (hipStream_t)stream), (hipStream_t)stream,
                      "enc_cache_fork");
}

enc_status enc_cache_shared(const enc_cache *c, const int32_t *d_seqs, uint32_t batch, const int32_t *d_starts,
                            uint32_t groups, int32_t *d_shared, void *stream) {
  set_error(ENC_OK, "%s", "");
  const enc_status st = check_cache(c);
  if (st != ENC_OK) return st;
  if (!groups) return ENC_OK;
  if (groups > (1u << 20) || batch > 0x7FFFFFFFu) return unsupported("more than 2^20 groups, or batch above 2^31 - 1");
  if ((batch && !d_seqs) || !d_starts || !d_shared || !aligned(d_seqs, 4) || !aligned(d_starts, 4) || !aligned(d_shared, 4))
    return invalid("seqs, starts or shared NULL or misaligned");
  return after_launch(launch_cache_shared(*c, d_seqs, batch, d_starts, groups, d_shared, (hipStream_t)stream),
                      (hipStream_t)stream, "enc_cache_shared");
}

enc_status enc_cache_truncate(const enc_cache *c, const int32_t *d_seqs, const int32_t *d_new_lens, uint32_t count,
                              void *stream) {
  set_error(ENC_OK, "%s", "");
  const enc_status st = check_cache(c);
  if (st != ENC_OK) return st;
  if (!count) return ENC_OK;
  if (count > 65535) return unsupported("more than 65535 sequences");
  if (!d_seqs || !d_new_lens || !aligned(d_seqs, 4) || !aligned(d_new_lens, 4))
    return invalid("seqs or new_lens NULL or misaligned");
  return after_launch(launch_cache_truncate(*c, d_seqs, d_new_lens, count, (hipStream_t)stream), (hipStream_t)stream,
                      "enc_cache_truncate");
}

}  // extern "C"
