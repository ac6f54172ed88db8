// Eviction from a paged cache by accumulated attention weight ("feat(gemma4): paged KV serving
// across both attention families", Description: one pool per family, pages shared by every layer
// of it, so every layer and head of a request keeps the same number of keys).
//
// A segment is one (layer, request, KV head); its n keys sit in slots [0, n) of the request's
// page list. It keeps n' = min(n, budget): the keys whose position is below num_sink or among
// the last num_recent first, then the largest masses, equal masses by lower slot.
//
//   select  finds the n'-th largest key by a radix descent over the masses' order-preserving bit
//           patterns (8 bits a pass) and writes, for each slot below n', the slot whose key will
//           sit there: kept keys already below n' stay, and the kept keys at or past n' fill the
//           holes below it, both in slot order. At most min(n', n - n') rows move (one per head
//           when a step evicts one key), and sources and destinations are disjoint, so
//   apply   moves rows in place with no staging and in any order.
#include "pg_internal.h"

#include <math.h>

namespace pg {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kWarps = kSelThreads / 32;

struct Seg {
  int32_t layer, r, g;
  int32_t kvp0, kvp1, n, keep, pos_end;
};
__device__ __forceinline__ Seg load_seg(const EvictArgs& a, int64_t s) {
  Seg q;
  const int32_t Hkv = a.pool.num_kv_heads;
  q.g = (int32_t)(s % Hkv);
  q.r = (int32_t)(s / Hkv % a.plan.num_req);
  q.layer = (int32_t)(s / Hkv / a.plan.num_req);
  q.kvp0 = a.plan.kv_page_indptr[q.r];
  q.kvp1 = a.plan.kv_page_indptr[q.r + 1];
  q.n = (q.kvp1 - q.kvp0 - 1) * a.pool.page_size + a.plan.last_page_len[q.r];
  q.keep = min(q.n, a.budget);
  q.pos_end = a.plan.start_pos[q.r] + (a.plan.qo_indptr[q.r + 1] - a.plan.qo_indptr[q.r]);
  return q;
}
__device__ __forceinline__ int32_t page_of(const EvictArgs& a, const Seg& q, int32_t slot) {
  const int32_t pidx = q.kvp0 + slot / a.pool.page_size;
  const int32_t p = (pidx < q.kvp1 && pidx < a.plan.num_page_ids) ? a.plan.page_ids[pidx] : -1;
  return p >= 0 && p < a.pool.num_pages ? p : -1;
}
__device__ __forceinline__ int64_t stat_at(const EvictArgs& a, const Seg& q, int32_t page, int32_t slot) {
  return (int64_t)q.layer * a.stats.stride_layer +
         ((int64_t)page * a.pool.num_kv_heads + q.g) * a.pool.page_size + slot % a.pool.page_size;
}
// Order of the keys as unsigned numbers: larger is kept first. Protected positions are above
// every mass; NaN counts as -inf; -0 as +0.
__device__ __forceinline__ uint32_t order_of(const EvictArgs& a, const Seg& q, int32_t slot) {
  const int32_t page = page_of(a, q, slot);
  if (page < 0) {
    atomicOr(a.status, kStatusBounds);
    return 0u;
  }
  const int64_t at = stat_at(a, q, page, slot);
  const int32_t pos = a.stats.pos[at];
  if (pos < a.num_sink || (int64_t)pos >= (int64_t)q.pos_end - a.num_recent) return 0xFFFFFFFFu;
  float m = a.stats.mass[at];
  if (isnan(m)) m = -INFINITY;
  const uint32_t b = __float_as_uint(m + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Inclusive counts over the block of a predicate, in thread order; *total the block's sum.
__device__ __forceinline__ int32_t block_rank(bool v, int32_t* warp_sum, int32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t b = __ballot_sync(0xffffffffu, v);
  if (lane == 0) warp_sum[warp] = __popc(b);
  __syncthreads();
  int32_t before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    const int32_t c = warp_sum[w];
    before += w < warp ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + __popc(b & ((2u << lane) - 1u));
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ int32_t warp_sum[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int32_t s_need;
  const Seg q = load_seg(a, blockIdx.x);
  int32_t* src = a.src + (int64_t)blockIdx.x * a.budget;
  const int tid = threadIdx.x;
  for (int32_t s = q.keep + tid; s < a.budget; s += kSelThreads) src[s] = -1;
  if (q.keep == q.n) {
    for (int32_t s = tid; s < q.keep; s += kSelThreads) src[s] = s;
    return;
  }
  // ---- the order value of the keep-th key, and how many of its equals are kept
  uint32_t prefix = 0u;
  int32_t need = q.keep;  // keys still to take among those matching the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    for (int32_t s = tid; s < q.n; s += kSelThreads) {
      const uint32_t o = order_of(a, q, s);
      if (shift == 24 || (o >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(o >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      int32_t left = need;
      int b = 255;
      while (b > 0 && (int32_t)hist[b] < left) left -= (int32_t)hist[b--];
      s_prefix = prefix | ((uint32_t)b << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  // ---- kept keys at or past the new length, in slot order, listed in src[0, movers)
  int32_t ties = 0, ties_low = 0, movers = 0;
  for (int32_t s0 = 0; s0 < q.n; s0 += kSelThreads) {
    const int32_t s = s0 + tid;
    const uint32_t o = s < q.n ? order_of(a, q, s) : 0u;
    const bool tie = s < q.n && o == prefix;
    int32_t total;
    const int32_t t = block_rank(tie, warp_sum, &total);
    const bool kept = s < q.n && (o > prefix || (tie && ties + t <= need));
    ties += total;
    ties_low += __syncthreads_count(tie && s < q.keep);
    const bool mover = kept && s >= q.keep;
    const int32_t k = block_rank(mover, warp_sum, &total);
    if (mover) src[movers + k - 1] = s;
    movers += total;
  }
  __syncthreads();
  // ---- holes below the new length, from the last block of slots to the first: a block reads
  // the list entries of its holes (a hole's rank is at most its slot) before it writes its slots
  int32_t holes_left = movers, ties_left = ties_low;
  for (int32_t s0 = (q.keep - 1) / kSelThreads * kSelThreads; s0 >= 0; s0 -= kSelThreads) {
    const int32_t s = s0 + tid;
    const bool in = s < q.keep;
    const uint32_t o = in ? order_of(a, q, s) : 0u;
    const bool tie = in && o == prefix;
    int32_t total;
    const int32_t t = block_rank(tie, warp_sum, &total);
    ties_left -= total;
    const bool hole = in && !(o > prefix || (tie && ties_left + t <= need));
    const int32_t k = block_rank(hole, warp_sum, &total);
    holes_left -= total;
    const int32_t from = hole ? src[holes_left + k - 1] : s;
    __syncthreads();
    if (in) src[s] = from;
    __syncthreads();
  }
}

// One warp per 32 kept slots: the slots whose key comes from elsewhere are copied one by one,
// the row's 16-byte pieces spread over the lanes.
constexpr int kApplyThreads = 256;
__global__ void __launch_bounds__(kApplyThreads) evict_apply_kernel(EvictArgs a, int32_t groups) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5);
  const int64_t segs = (int64_t)a.num_layers * a.plan.num_req * a.pool.num_kv_heads;
  const int64_t seg = w / groups;
  if (seg >= segs) return;
  const Seg q = load_seg(a, seg);
  const int32_t slot = (int32_t)(w % groups) * 32 + lane;
  int32_t from = slot;
  if (slot < q.keep) from = a.src[seg * a.budget + slot];
  bool move = from >= 0 && from != slot;
  int32_t fp = -1, tp = -1;
  if (move) {
    // a source below the new length, or past the keys, is not one that select gives
    fp = from >= q.keep && from < q.n ? page_of(a, q, from) : -1;
    tp = page_of(a, q, slot);
    if (fp < 0 || tp < 0) {
      atomicOr(a.status, kStatusBounds);
      move = false;
    }
  }
  if (move) {
    const int64_t x = stat_at(a, q, fp, from), y = stat_at(a, q, tp, slot);
    a.stats.mass[y] = a.stats.mass[x];
    a.stats.pos[y] = a.stats.pos[x];
  }
  const int32_t D = a.pool.head_dim, ps = a.pool.page_size;
  __nv_bfloat16* base = a.pool.layer_base + (int64_t)q.layer * a.pool_stride_layer +
                        (int64_t)q.g * a.pool.stride_head;
  for (uint32_t b = __ballot_sync(0xffffffffu, move); b; b &= b - 1) {
    const int l = __ffs(b) - 1;
    const int32_t f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, slot, l);
    const int32_t fpage = __shfl_sync(0xffffffffu, fp, l), tpage = __shfl_sync(0xffffffffu, tp, l);
    const __nv_bfloat16* x = base + (int64_t)fpage * a.pool.stride_page + (int64_t)(f % ps) * D;
    __nv_bfloat16* y = base + (int64_t)tpage * a.pool.stride_page + (int64_t)(t % ps) * D;
    for (int32_t c = lane * 8; c < D; c += 256) {
      const uint4 k = *reinterpret_cast<const uint4*>(x + c);
      const uint4 v = *reinterpret_cast<const uint4*>(x + a.pool.stride_kv + c);
      *reinterpret_cast<uint4*>(y + c) = k;
      *reinterpret_cast<uint4*>(y + a.pool.stride_kv + c) = v;
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t stream) {
  const int64_t segs = (int64_t)a.num_layers * a.plan.num_req * a.pool.num_kv_heads;
  if (segs == 0) return cudaSuccess;
  evict_select_kernel<<<(unsigned)segs, kSelThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_evict_apply(const EvictArgs& a, cudaStream_t stream) {
  const int64_t segs = (int64_t)a.num_layers * a.plan.num_req * a.pool.num_kv_heads;
  const int32_t keep = a.max_keys < a.budget ? a.max_keys : a.budget;
  if (segs == 0 || keep == 0) return cudaSuccess;
  const int32_t groups = (keep + 31) / 32;
  const int64_t blocks = (segs * groups + kApplyThreads / 32 - 1) / (kApplyThreads / 32);
  evict_apply_kernel<<<(unsigned)blocks, kApplyThreads, 0, stream>>>(a, groups);
  count_launch();
  return cudaGetLastError();
}

}  // namespace pg
