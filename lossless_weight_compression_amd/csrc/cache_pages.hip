// cache_pages.hip -- pages of a key/value cache: append accepted rows (with
// copy on write of a shared last page), share all pages with a fork, free the
// pages past a new end.
//
// The bookkeeping is integers only, so its results do not depend on order:
// free pages are those whose count is 0 when the call begins, and the r-th
// page that the call's sequences need (in the order of the call) is the r-th
// free one. A commit is two kernels. The first, one workgroup, checks every
// number it was given, counts needs and free pages and either updates the
// table, the counts and the lengths or leaves everything as it was. The
// second moves the rows, and is bound by HBM traffic: a workgroup per
// (sequence, plane, slice), 16 bytes a lane.
//
// Measured (us on the device): one sequence, 64 planes of 2048-byte rows: plan
// 4.1, move 2.9; 64 sequences of 32 nodes, 16 planes (65 MB): plan 8 to 9, move
// 15, 4.3 TB/s; 16 forks of one prompt that then append, copying 63 rows of their
// last page in 16 planes (71 MB): fork 2.6, plan 8.0, move 10.
//
// The plan counts the free pages of the whole pool, 64 counts a wave at a time,
// and then walks them again up to the last one needed: a call that needs one
// page takes 1 us more with 10000 pages than with 100, 12 with 100000 (32 if
// the first free one comes after nine tenths of them), 142 (320) with a million.
#include "step_common.h"

namespace enc {
namespace {

constexpr uint32_t kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr uint32_t kCopyThreads = 256;

enum { kBadSeq = -1, kBadPath = -2, kPastEnd = -3, kBadTable = -4 };

__device__ __forceinline__ uint32_t wave_scan_incl(uint32_t v, uint32_t lane) {
  for (uint32_t o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive sum over the workgroup; total to every thread.
__device__ __forceinline__ uint32_t block_scan_excl(uint32_t v, uint32_t *sums, uint32_t &total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t incl = wave_scan_incl(v, lane);
  __syncthreads();
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (uint32_t w = 0; w < kPlanWaves; ++w) {
    const uint32_t t = sums[w];
    if (w < wave) before += t;
    all += t;
  }
  total = all;
  return before + incl - v;
}

// The new pages sequence b needs: its partly filled last page if somebody
// else holds that too, and every page that its new rows reach and it lacks.
struct Need {
  int32_t seq, len, rows, last;   // last: the shared page to copy, or -1
  uint32_t pages;
  int32_t error;
};

__device__ __forceinline__ Need need_of(const CommitArgs &k, uint32_t b) {
  Need n;
  n.seq = k.seqs[b];
  n.rows = k.count[b];
  n.len = 0;
  n.last = -1;
  n.pages = 0;
  n.error = 0;
  if ((uint32_t)n.seq >= k.c.max_seqs) { n.error = kBadSeq; return n; }
  if (n.rows < 0 || (uint32_t)n.rows > k.nodes) { n.error = kBadPath; return n; }
  n.len = k.c.d_lens[n.seq];
  const uint64_t room = (uint64_t)k.c.max_pages * k.c.page_size;
  if (n.len < 0 || (uint64_t)n.len > room) { n.error = kBadTable; return n; }
  if ((uint64_t)n.len + n.rows > room) { n.error = kPastEnd; return n; }
  if (n.rows == 0) return n;
  const int32_t *row = k.c.d_table + (uint64_t)n.seq * k.c.max_pages;
  const uint32_t p0 = k.page.quot(n.len), p1 = k.page.quot(n.len + n.rows - 1);
  const bool partly = p0 * k.c.page_size != (uint32_t)n.len;
  for (uint32_t p = p0; p <= p1; ++p) {
    const int32_t e = row[p];
    if (partly && p == p0) {
      if ((uint32_t)e >= k.c.n_pages) { n.error = kBadTable; return n; }
      const int32_t refs = k.c.d_refs[e];
      if (refs < 1) { n.error = kBadTable; return n; }   // held, yet free for others
      if (refs > 1) {
        n.last = e;
        ++n.pages;
      }
    } else {
      if (e != -1) { n.error = kBadTable; return n; }
      ++n.pages;
    }
  }
  return n;
}

__global__ __launch_bounds__(kPlanThreads) void k_commit_plan(CommitArgs k) {
  __shared__ uint32_t sums[kPlanWaves];
  __shared__ int32_t error;
  __shared__ uint32_t wave_free[kPlanWaves];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) error = 0;
  __syncthreads();

  for (uint64_t i = tid; i < (uint64_t)k.batch * k.nodes; i += kPlanThreads) {
    const uint32_t b = (uint32_t)(i / k.nodes), j = (uint32_t)(i - (uint64_t)b * k.nodes);
    if ((int32_t)j < k.count[b] && (uint32_t)k.path[i] >= k.nodes) atomicMin(&error, (int32_t)kBadPath);
  }
  uint32_t need = 0;
  for (uint32_t b0 = 0; b0 < k.batch; b0 += kPlanThreads) {
    const uint32_t b = b0 + tid;
    Need n;
    n.pages = 0;
    if (b < k.batch) {
      n = need_of(k, b);
      if (n.error) atomicMin(&error, n.error);
    }
    uint32_t all;
    const uint32_t before = block_scan_excl(n.pages, sums, all);
    if (b < k.batch) {
      k.first[b] = (int32_t)(need + before);
      k.info[4 * b + 0] = n.len;
      k.info[4 * b + 1] = n.rows;
      k.info[4 * b + 2] = n.last;
      k.info[4 * b + 3] = -1;
    }
    need += all;
  }
  __syncthreads();

  // Free pages: each wave counts those of its range, then, knowing how many
  // lie before it, ranks the ones the call needs.
  const uint32_t range = ((k.c.n_pages + kPlanWaves - 1) / kPlanWaves + 63) & ~63u;
  const uint32_t g0 = min(wave * range, k.c.n_pages), g1 = min(g0 + range, k.c.n_pages);
  uint32_t found = 0;
  if (need && !error) {
    uint32_t mine = 0;
    for (uint32_t g = g0 + lane; g < g1; g += 64) mine += k.c.d_refs[g] == 0;
    for (uint32_t o = 32; o; o >>= 1) mine += __shfl_xor(mine, o);
    if (lane == 0) wave_free[wave] = mine;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < kPlanWaves; ++w) {
      if (w < wave) before += wave_free[w];
      found += wave_free[w];
    }
    if (found >= need) {
      for (uint32_t g = g0; g < g1 && before < need; g += 64) {
        const bool is_free = g + lane < g1 && k.c.d_refs[g + lane] == 0;
        const uint64_t m = __ballot(is_free);
        const uint32_t rank = before + __popcll(m & ((1ull << lane) - 1));
        if (is_free && rank < need) k.pick[rank] = (int32_t)(g + lane);
        before += __popcll(m);
      }
    }
  }
  __syncthreads();
  const int32_t status = error ? error : found < need ? (int32_t)(need - found) : 0;
  if (tid == 0) *k.status = status;
  if (status) {   // nothing to move
    for (uint32_t b = tid; b < k.batch; b += kPlanThreads) k.info[4 * b + 3] = -1;
    for (uint64_t i = tid; i < (uint64_t)k.batch * k.nodes; i += kPlanThreads) k.to[i] = -1;
    return;
  }

  for (uint32_t b = tid; b < k.batch; b += kPlanThreads) {
    const int32_t len = k.info[4 * b], rows = k.info[4 * b + 1];
    if (rows == 0) continue;
    const uint32_t seq = (uint32_t)k.seqs[b];
    const int32_t last = k.info[4 * b + 2];
    int32_t *row = k.c.d_table + (uint64_t)seq * k.c.max_pages;
    const uint32_t p0 = k.page.quot(len), p1 = k.page.quot(len + rows - 1);
    uint32_t next = (uint32_t)k.first[b];
    for (uint32_t p = p0; p <= p1; ++p) {
      // the page's count may have changed since: a page that several sequences
      // of this call share is left by each of them
      const bool leave = p == p0 && last >= 0;
      if (row[p] >= 0 && !leave) continue;
      const int32_t got = k.pick[next++];
      row[p] = got;
      k.c.d_refs[got] = 1;
      if (leave) {
        atomicSub(&k.c.d_refs[last], 1);
        k.info[4 * b + 3] = got;
      }
    }
    k.c.d_lens[seq] = len + rows;
  }
  __syncthreads();
  // where each accepted row goes
  for (uint64_t i = tid; i < (uint64_t)k.batch * k.nodes; i += kPlanThreads) {
    const uint32_t b = (uint32_t)(i / k.nodes), j = (uint32_t)(i - (uint64_t)b * k.nodes);
    int32_t to = -1;
    if ((int32_t)j < k.info[4 * b + 1]) {
      const uint32_t t = (uint32_t)k.info[4 * b] + j, p = k.page.quot(t);
      to = (int32_t)((uint32_t)k.c.d_table[(uint64_t)(uint32_t)k.seqs[b] * k.c.max_pages + p] * k.c.page_size +
                     (t - p * k.c.page_size));
    }
    k.to[i] = to;
  }
}

// One (sequence, plane)'s rows: a slot for every node of the tree (empty past
// the accepted ones), in `node_groups` workgroups, one slot to a thread; then
// the filled rows of a page that is left, by the other workgroups in turn. A
// slot is `lanes` threads wide, 16 bytes each. The loads in flight come from
// many small workgroups: with four slots to a thread it took twice as long.
__global__ __launch_bounds__(kCopyThreads) void k_commit_move(CommitArgs k, FastDiv lanes, uint32_t slots,
                                                              uint32_t node_groups) {
  const uint32_t b = blockIdx.x;
  const uint64_t plane = blockIdx.y;
  const uint32_t ps = k.c.page_size, row_bytes = k.c.row_bytes;
  uint8_t *base = static_cast<uint8_t *>(k.c.d_data) + plane * k.c.plane_stride;
  const uint32_t in = lanes.quot(threadIdx.x), lane = threadIdx.x - in * lanes.d;   // slot of the workgroup, place in it
  if (in >= slots) return;
  if (blockIdx.z < node_groups) {
    const uint32_t slot = blockIdx.z * slots + in;
    if (slot >= k.nodes) return;
    const int32_t to = k.to[(uint64_t)b * k.nodes + slot], node = k.path[(uint64_t)b * k.nodes + slot];
    if (to < 0) return;
    const uint8_t *src = k.draft + plane * k.draft_plane + (uint64_t)b * k.draft_seq + (uint64_t)(uint32_t)node * row_bytes;
    uint8_t *dst = base + (uint64_t)(uint32_t)to * row_bytes;
    for (uint32_t o = lane * 16; o < row_bytes; o += lanes.d * 16)
      store_nt16(dst + o, *reinterpret_cast<const uint4 *>(src + o));
    return;
  }
  const int32_t len = k.info[4 * b], from = k.info[4 * b + 2], to = k.info[4 * b + 3];
  if (to < 0) return;
  const uint32_t filled = (uint32_t)len - k.page.quot((uint32_t)len) * ps;
  const uint32_t step = (gridDim.z - node_groups) * slots;
  for (uint32_t r = (blockIdx.z - node_groups) * slots + in; r < filled; r += step) {
    const uint8_t *src = base + ((uint64_t)(uint32_t)from * ps + r) * row_bytes;
    uint8_t *dst = base + ((uint64_t)(uint32_t)to * ps + r) * row_bytes;
    for (uint32_t o = lane * 16; o < row_bytes; o += lanes.d * 16)
      store_nt16(dst + o, *reinterpret_cast<const uint4 *>(src + o));
  }
}

__global__ __launch_bounds__(kCopyThreads) void k_fork(enc_cache c, const int32_t *src, const int32_t *dst) {
  const uint32_t i = blockIdx.y, p = blockIdx.x * kCopyThreads + threadIdx.x;
  const uint32_t s = (uint32_t)src[i], d = (uint32_t)dst[i];
  if (s >= c.max_seqs || d >= c.max_seqs || s == d) return;
  if (p < c.max_pages) {
    const int32_t gain = c.d_table[(uint64_t)s * c.max_pages + p];
    int32_t *at = c.d_table + (uint64_t)d * c.max_pages + p;
    const int32_t loss = *at;
    if (loss != gain) {
      if ((uint32_t)loss < c.n_pages) atomicSub(&c.d_refs[loss], 1);
      if ((uint32_t)gain < c.n_pages) atomicAdd(&c.d_refs[gain], 1);
      *at = gain;
    }
  }
  if (p == 0) c.d_lens[d] = c.d_lens[s];
}

// Lengths may be written before another workgroup of the same sequence reads
// them: the smaller of old and new length is the same either way.
__global__ __launch_bounds__(kCopyThreads) void k_truncate(enc_cache c, const int32_t *seqs, const int32_t *lens) {
  const uint32_t i = blockIdx.y, p = blockIdx.x * kCopyThreads + threadIdx.x;
  const uint32_t s = (uint32_t)seqs[i];
  if (s >= c.max_seqs) return;
  const int32_t keep = max(0, min(c.d_lens[s], lens[i]));
  if (p < c.max_pages && (uint64_t)p * c.page_size >= (uint32_t)keep) {
    int32_t *at = c.d_table + (uint64_t)s * c.max_pages + p;
    const int32_t e = *at;
    if (e >= 0) {
      if ((uint32_t)e < c.n_pages) atomicSub(&c.d_refs[e], 1);
      *at = -1;
    }
  }
  if (p == 0) c.d_lens[s] = keep;
}

}  // namespace

hipError_t launch_cache_commit(const CommitArgs &k, hipStream_t s) {
  hipLaunchKernelGGL(k_commit_plan, dim3(1), dim3(kPlanThreads), 0, s, k);
  const uint32_t per = k.c.row_bytes / 16, lanes = per < kCopyThreads ? per : kCopyThreads, slots = kCopyThreads / lanes;
  const uint32_t node_groups = (k.nodes + slots - 1) / slots, copy_groups = (k.c.page_size + slots - 1) / slots;
  hipLaunchKernelGGL(k_commit_move, dim3(k.batch, k.c.n_planes, node_groups + (copy_groups < 32 ? copy_groups : 32)),
                     dim3(kCopyThreads), 0, s, k, FastDiv::of(lanes), slots, node_groups);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const enc_cache &c, const int32_t *src, const int32_t *dst, uint32_t pairs,
                             hipStream_t s) {
  hipLaunchKernelGGL(k_fork, dim3((c.max_pages + kCopyThreads - 1) / kCopyThreads, pairs), dim3(kCopyThreads), 0, s,
                     c, src, dst);
  return hipGetLastError();
}

hipError_t launch_cache_truncate(const enc_cache &c, const int32_t *seqs, const int32_t *lens, uint32_t count,
                                 hipStream_t s) {
  hipLaunchKernelGGL(k_truncate, dim3((c.max_pages + kCopyThreads - 1) / kCopyThreads, count), dim3(kCopyThreads), 0,
                     s, c, seqs, lens);
  return hipGetLastError();
}

}  // namespace enc
