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

struct Seg {
  int32_t layer, r, g;
  int32_t kvp0, kvp1, n, keep;
};
__device__ __forceinline__ Seg load_seg(const EvictArgs& a, int32_t s) {
  Seg q;
  const int32_t Hkv = a.pool.num_kv_heads;
  q.g = s % Hkv;
  q.r = s / Hkv % a.plan.num_req;
  q.layer = s / Hkv / a.plan.num_req;
  q.kvp0 = a.plan.kv_page_indptr[q.r];
  q.kvp1 = a.plan.kv_page_indptr[q.r + 1];
  q.n = (q.kvp1 - q.kvp0 - 1) * a.pool.page_size + a.plan.last_page_len[q.r];
  q.keep = min(q.n, a.budget);
  return q;
}
// slot / page_size by the multiplier that the host works out (set_page_divisor)
__device__ __forceinline__ int32_t page_index(const EvictArgs& a, int32_t slot) {
  return a.page_mul ? (int32_t)(__umulhi((uint32_t)slot, a.page_mul) >> a.page_shift) : slot;
}
__device__ __forceinline__ int32_t page_offset(const EvictArgs& a, int32_t slot) {
  return slot - page_index(a, slot) * a.pool.page_size;
}
__device__ __forceinline__ int32_t page_of(const EvictArgs& a, const Seg& q, int32_t slot) {
  const int32_t pidx = q.kvp0 + page_index(a, slot);
  const int32_t p = (pidx < q.kvp1 && pidx < a.plan.num_page_ids) ? a.plan.page_ids[pidx] : -1;
  return p >= 0 && p < a.pool.num_pages ? p : -1;
}
__device__ __forceinline__ int64_t stat_at(const EvictArgs& a, const Seg& q, int32_t page, int32_t slot) {
  return (int64_t)q.layer * a.stats.stride_layer +
         ((int64_t)page * a.pool.num_kv_heads + q.g) * a.pool.page_size + page_offset(a, slot);
}
// First protected position of the segment's last ones.
__device__ __forceinline__ int64_t recent_from(const EvictArgs& a, const Seg& q) {
  const int32_t end = a.plan.start_pos[q.r] + (a.plan.qo_indptr[q.r + 1] - a.plan.qo_indptr[q.r]);
  return (int64_t)end - a.num_recent;
}
// Order of a key as an unsigned number, larger kept first: protected positions above every mass,
// NaN as -inf, -0 as +0. 0 is no key, 1 a key on a page that is out of range.
__device__ __forceinline__ uint32_t order_of(const EvictArgs& a, int64_t recent, int32_t pos, float m) {
  if (pos < a.num_sink || pos >= recent) return 0xFFFFFFFFu;
  if (isnan(m)) m = -INFINITY;
  const uint32_t b = __float_as_uint(m + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// ------------------------------------------------------------------ select
// One CTA (or a cluster of up to 8) per segment, its keys in registers: thread t of the segment
// holds slots [k t, k (t + 1)), k <= KPT the segment's share of them in groups of four, so slot
// order is thread order and every rank below is a bit count over the thread's 32-bit masks and one
// scan over the threads. Statistics are read four slots at a time where the pages and the arrays
// allow it (V4).
//
// The keep-th largest order value is built bit by bit from the top: a candidate stays when at
// least keep keys reach it, one count over the segment per bit (compares in registers, a warp
// reduction and one barrier: no histogram, so equal exponents cost nothing). The descent ends when
// exactly keep keys reach the candidate (then nothing ties), about 20 bits in for masses that
// differ; once 1024 keys or fewer share the bits so far, they are gathered and only they are
// counted (two a thread). Bound: a segment is read once (8 bytes a key), and the counts are two
// instructions per key and bit; with them one CTA on an SM covers the other's loads.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kGather = 2 * kSelThreads;  // keys gathered out of the segment: two a thread

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t peer(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Counts over the segment's threads. Buffers are used alternately, so one barrier a call is enough.
template <bool CL>
struct Counter {
  int32_t (*warp_sum)[kSelWarps];  // [2][warps]
  int2 (*cta_sum)[kMaxCluster];    // [2][ranks], in every CTA of the cluster
  int rank, ranks, phase;
  // over the cluster: the total, and the ranks before this one
  __device__ __forceinline__ int2 cluster(int2 v, int2* before) {
    const int lane = threadIdx.x & 31;
    if ((threadIdx.x >> 5) == 0 && lane < ranks) {
      const uint32_t to = peer(smem_u32(&cta_sum[phase][rank]), lane);
      asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(to), "r"(v.x), "r"(v.y) : "memory");
    }
    cluster_barrier();
    const int2 c = lane < ranks ? cta_sum[phase][lane] : make_int2(0, 0);
    before->x = __reduce_add_sync(0xffffffffu, lane < rank ? c.x : 0);
    before->y = __reduce_add_sync(0xffffffffu, lane < rank ? c.y : 0);
    return make_int2(__reduce_add_sync(0xffffffffu, c.x), __reduce_add_sync(0xffffffffu, c.y));
  }
  __device__ __forceinline__ int32_t total(int32_t v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) warp_sum[phase][warp] = v;
    __syncthreads();
    int32_t t = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_sum[phase][lane] : 0);
    if constexpr (CL) {
      int2 unused;
      t = cluster(make_int2(t, 0), &unused).x;
    }
    phase ^= 1;
    return t;
  }
  // two counts per thread (at most KPT each): the threads before this one, and the totals
  __device__ __forceinline__ int2 before(int32_t x, int32_t y, int2* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // packed in 16 bits each: a CTA holds at most 16,384 slots
    const uint32_t v = (uint32_t)x | (uint32_t)y << 16;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t w = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += w;
    }
    if (lane == 31) warp_sum[phase][warp] = (int32_t)incl;
    __syncthreads();
    const uint32_t w = lane < kSelWarps ? (uint32_t)warp_sum[phase][lane] : 0u;
    const uint32_t t = __reduce_add_sync(0xffffffffu, w);
    const uint32_t p = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u) + incl - v;
    int2 b = make_int2((int32_t)(p & 0xFFFFu), (int32_t)(p >> 16));
    *all = make_int2((int32_t)(t & 0xFFFFu), (int32_t)(t >> 16));
    if constexpr (CL) {
      int2 r;
      *all = cluster(*all, &r);
      b.x += r.x;
      b.y += r.y;
    }
    phase ^= 1;
    return b;
  }
};

template <int KPT, bool CL, bool V4>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(EvictArgs a, int32_t ranks) {
  // kept keys past the new length, by rank: at most half of the cluster's slots, spread over it
  constexpr int kList = kSelThreads * KPT / 2;
  __shared__ int32_t warp_sum[2][kSelWarps];
  __shared__ int2 cta_sum[2][kMaxCluster];
  extern __shared__ int32_t list[];
  const int32_t rank = CL ? (int32_t)(blockIdx.x % ranks) : 0;
  const int32_t seg = CL ? (int32_t)(blockIdx.x / ranks) : (int32_t)blockIdx.x;
  const Seg q = load_seg(a, seg);
  int32_t* src = a.src + (int64_t)seg * a.budget;
  const int tid = threadIdx.x;
  const int32_t step = CL ? kSelThreads * ranks : kSelThreads, first = rank * kSelThreads + tid;
  const bool fits = q.n <= kSelThreads * KPT * (CL ? ranks : 1);
  // every slot keeps its key until a hole below says otherwise
  if (!CL || q.keep == q.n || !fits)  // (a cluster that goes on does it below)
    for (int32_t s = first; s < a.budget; s += step) src[s] = s < q.keep ? s : -1;
  if (q.keep == q.n) return;  // (the whole cluster)
  if (!fits) {  // a plan that grew past its captured launch
    if (tid == 0) atomicOr(a.status, kStatusBounds);
    return;
  }
  if constexpr (CL) {
    // (the cluster's barriers order every slot before the holes); and every peer runs before its
    // shared memory is written
    for (int32_t s = first; s < a.budget; s += step) src[s] = s < q.keep ? s : -1;
    cluster_barrier();
  }
  const int64_t recent = recent_from(a, q);
  // the segment's slots in equal shares: groups of four (whole groups keep V4's vectors in a page)
  const int32_t threads = kSelThreads * (CL ? ranks : 1);
  const int32_t share = ((q.n + threads - 1) / threads + 3) & ~3;
  const int32_t s0 = (rank * kSelThreads + tid) * share;
  const int32_t s_end = min(q.n, s0 + share);
  uint32_t key[KPT];
  if constexpr (V4) {
    // four slots of one page at a time, all loads in flight before the first use
    constexpr int B = KPT < 16 ? KPT / 4 : 4;  // groups per batch
#pragma unroll
    for (int i0 = 0; i0 < KPT / 4; i0 += B) {
      int32_t page[B];
      int4 pos[B];
      float4 m[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int32_t s = s0 + 4 * (i0 + i);
        page[i] = s < s_end ? page_of(a, q, s) : -2;
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        pos[i] = make_int4(0, 0, 0, 0);
        m[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (page[i] >= 0) {
          const int64_t at = stat_at(a, q, page[i], s0 + 4 * (i0 + i));
          pos[i] = *reinterpret_cast<const int4*>(a.stats.pos + at);
          m[i] = *reinterpret_cast<const float4*>(a.stats.mass + at);
        }
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int32_t s = s0 + 4 * (i0 + i);
        const int32_t p4[4] = {pos[i].x, pos[i].y, pos[i].z, pos[i].w};
        const float m4[4] = {m[i].x, m[i].y, m[i].z, m[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          key[4 * (i0 + i) + e] = s + e >= s_end ? 0u : page[i] < 0 ? 1u : order_of(a, recent, p4[e], m4[e]);
        if (page[i] == -1) atomicOr(a.status, kStatusBounds);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int32_t s = s0 + i, page = s < s_end ? page_of(a, q, s) : -2;
      key[i] = page == -2 ? 0u : 1u;
      if (page >= 0) {
        const int64_t at = stat_at(a, q, page, s);
        key[i] = order_of(a, recent, a.stats.pos[at], a.stats.mass[at]);
      } else if (page == -1) {
        atomicOr(a.status, kStatusBounds);
      }
    }
  }
  Counter<CL> count{warp_sum, cta_sum, rank, ranks, 0};
  // ---- the keep-th largest order value
  uint32_t cut = 0u;
  int32_t reach = q.n, above = 0;  // keys from cut up, and from the end of its range (cut + 2^(bit + 1)) up
  int bit = 31;
  for (; bit >= 0; --bit) {
    if (!CL && reach - above <= kGather && bit >= 3) break;
    const uint32_t cand = cut | (1u << bit);
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < KPT; i += 4) {
      if (i < share)  // (uniform)
        c += (key[i] >= cand ? 1 : 0) + (key[i + 1] >= cand ? 1 : 0) + (key[i + 2] >= cand ? 1 : 0) +
             (key[i + 3] >= cand ? 1 : 0);
    }
    c = count.total(c);
    if (c >= q.keep) {
      cut = cand;
      reach = c;
    } else {
      above = c;
    }
    if (c == q.keep) {  // exactly the keys from cand up: no lower bit can matter
      bit = -1;
      break;
    }
  }
  if constexpr (!CL) {
    if (bit >= 0) {
      // the few keys of the range, two a thread
      const uint32_t top = bit == 31 ? 0xFFFFFFFFu : cut + ((1u << (bit + 1)) - 1u);  // the range's last
      int32_t mine = 0;
#pragma unroll
      for (int i = 0; i < KPT; ++i) mine += key[i] >= cut && key[i] <= top && key[i] != 0u ? 1 : 0;
      int2 all;
      int32_t at = count.before(mine, 0, &all).x;
#pragma unroll
      for (int i = 0; i < KPT; ++i)
        if (key[i] >= cut && key[i] <= top && key[i] != 0u) list[at++] = (int32_t)key[i];
      __syncthreads();
      uint32_t few[kGather / kSelThreads];
#pragma unroll
      for (int i = 0; i < kGather / kSelThreads; ++i) {
        const int32_t x = tid + i * kSelThreads;
        few[i] = x < all.x ? (uint32_t)list[x] : 0u;
      }
      for (; bit >= 0; --bit) {
        const uint32_t cand = cut | (1u << bit);
        int32_t c = 0;
#pragma unroll
        for (int i = 0; i < kGather / kSelThreads; ++i) c += few[i] >= cand ? 1 : 0;
        c = above + count.total(c);
        if (c >= q.keep) cut = cand;
        if (c == q.keep) break;
      }
    }
  }
  // ---- kept slots: above the cut, and the lowest of those at it
  uint32_t kept = 0u, tie = 0u;
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    kept |= key[i] > cut ? 1u << i : 0u;
    tie |= key[i] == cut ? 1u << i : 0u;
  }
  int2 all;
  const int2 t = count.before(__popc(kept), __popc(tie), &all);
  for (int32_t left = q.keep - all.x - t.y; left > 0 && tie; --left) {
    kept |= tie & (0u - tie);
    tie &= tie - 1u;
  }
  // ---- movers (kept, at or past the new length) and holes (not kept, below it)
  const int32_t low = min(max(q.keep - s0, 0), max(s_end - s0, 0));  // this thread's slots below the new length
  const uint32_t mask = low >= 32 ? 0xFFFFFFFFu : (1u << low) - 1u;
  uint32_t mover = kept & ~mask, hole = ~kept & mask;
  const int2 at = count.before(__popc(mover), __popc(hole), &all);
  for (int32_t k = at.x; mover; mover &= mover - 1u, ++k) {
    const int32_t s = s0 + __ffs(mover) - 1;
    if constexpr (CL)
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer(smem_u32(list + k % kList), k / kList)), "r"(s)
                   : "memory");
    else
      list[k] = s;
  }
  if constexpr (CL) cluster_barrier();
  else __syncthreads();
  for (int32_t k = at.y; hole; hole &= hole - 1u, ++k) {
    int32_t from;
    if constexpr (CL)
      asm volatile("ld.shared::cluster.s32 %0, [%1];"
                   : "=r"(from)
                   : "r"(peer(smem_u32(list + k % kList), k / kList))
                   : "memory");
    else
      from = list[k];
    src[s0 + __ffs(hole) - 1] = from;
  }
  if constexpr (CL) cluster_barrier();  // the peers have read this CTA's list
}

// Segments longer than a cluster's registers (131,072 keys): one CTA, the keys read again for
// each of four 8-bit histogram passes and the two ranking passes.
constexpr int kLongThreads = 1024;
constexpr int kLongWarps = kLongThreads / 32;
__device__ __forceinline__ uint32_t order_at(const EvictArgs& a, const Seg& q, int64_t recent, int32_t slot) {
  const int32_t page = page_of(a, q, slot);
  if (page < 0) {
    atomicOr(a.status, kStatusBounds);
    return 1u;
  }
  const int64_t at = stat_at(a, q, page, slot);
  return order_of(a, recent, a.stats.pos[at], a.stats.mass[at]);
}
// Inclusive counts over the block of a predicate, in thread order; *total the block's sum.
__device__ __forceinline__ int32_t block_rank(bool v, int32_t* warp_sum, int32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t b = __ballot_sync(0xffffffffu, v);
  if (lane == 0) warp_sum[warp] = __popc(b);
  __syncthreads();
  int32_t before = 0, all = 0;
  for (int w = 0; w < kLongWarps; ++w) {
    const int32_t c = warp_sum[w];
    before += w < warp ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + __popc(b & ((2u << lane) - 1u));
}

__global__ void __launch_bounds__(kLongThreads) evict_select_long_kernel(EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ int32_t warp_sum[kLongWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int32_t s_need;
  const Seg q = load_seg(a, (int32_t)blockIdx.x);
  const int64_t recent = recent_from(a, q);
  int32_t* src = a.src + (int64_t)blockIdx.x * a.budget;
  const int tid = threadIdx.x;
  for (int32_t s = q.keep + tid; s < a.budget; s += kLongThreads) src[s] = -1;
  if (q.keep == q.n) {
    for (int32_t s = tid; s < q.keep; s += kLongThreads) src[s] = s;
    return;
  }
  // ---- the order value of the keep-th key, and how many of its equals are kept
  uint32_t prefix = 0u;
  int32_t need = q.keep;  // keys still to take among those matching the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kLongThreads) hist[i] = 0u;
    __syncthreads();
    for (int32_t s = tid; s < q.n; s += kLongThreads) {
      const uint32_t o = order_at(a, q, recent, s);
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
  for (int32_t s0 = 0; s0 < q.n; s0 += kLongThreads) {
    const int32_t s = s0 + tid;
    const uint32_t o = s < q.n ? order_at(a, q, recent, s) : 0u;
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
  for (int32_t s0 = (q.keep - 1) / kLongThreads * kLongThreads; s0 >= 0; s0 -= kLongThreads) {
    const int32_t s = s0 + tid;
    const bool in = s < q.keep;
    const uint32_t o = in ? order_at(a, q, recent, s) : 0u;
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

// ------------------------------------------------------------------ apply
// A block takes 1024 kept slots of one segment, a warp 128 of them, four a lane: it lists the
// slots whose key comes from elsewhere, then moves them four at a time, each row's 16-byte pieces
// spread over the lanes (at head_dim 512 a lane has 16 loads in flight), so the moves of a warp
// wait for memory once per four. Bound: 4 D bytes read and written per move, and the map read.
constexpr int kApplyThreads = 256, kApplySlots = 1024, kMoves = 4;
template <int D>
__global__ void __launch_bounds__(kApplyThreads) evict_apply_kernel(EvictArgs a, int32_t blocks_per_seg) {
  __shared__ int2 s_move[kApplyThreads / 32][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t seg = (int32_t)blockIdx.x / blocks_per_seg;
  const int32_t t0 = ((int32_t)blockIdx.x % blocks_per_seg) * kApplySlots + warp * 128 + lane;
  const int32_t* src = a.src + (int64_t)seg * a.budget;
  int32_t from[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) from[i] = t0 + 32 * i < a.budget ? src[t0 + 32 * i] : -1;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= from[i] >= 0 && from[i] != t0 + 32 * i;
  if (!__any_sync(0xffffffffu, any)) return;
  const Seg q = load_seg(a, seg);
  // rows (page * page_size + offset) of each move, listed by the warp
  int32_t count = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t to = t0 + 32 * i;
    bool move = from[i] >= 0 && from[i] != to;
    int32_t fp = -1, tp = -1;
    if (move) {
      // a target past the new length, or a source that select does not give, is not followed
      fp = to < q.keep && from[i] >= q.keep && from[i] < q.n ? page_of(a, q, from[i]) : -1;
      tp = to < q.keep ? page_of(a, q, to) : -1;
      if (fp < 0 || tp < 0) {
        atomicOr(a.status, kStatusBounds);
        move = false;
      }
    }
    const uint32_t b = __ballot_sync(0xffffffffu, move);
    if (move) {
      const int64_t x = stat_at(a, q, fp, from[i]), y = stat_at(a, q, tp, to);
      a.stats.mass[y] = a.stats.mass[x];
      a.stats.pos[y] = a.stats.pos[x];
      s_move[warp][count + __popc(b & ((1u << lane) - 1u))] = make_int2(from[i], to);
    }
    count += __popc(b);
  }
  __syncwarp();
  __nv_bfloat16* base = a.pool.layer_base + (int64_t)q.layer * a.pool_stride_layer +
                        (int64_t)q.g * a.pool.stride_head + lane * 8;
  auto row = [&](int32_t slot) {
    return base + (int64_t)page_of(a, q, slot) * a.pool.stride_page + (int64_t)page_offset(a, slot) * D;
  };
  constexpr int P = D / 256;  // 16-byte pieces of a row per lane
  for (int32_t i0 = 0; i0 < count; i0 += kMoves) {
    uint4 v[kMoves][2 * P];
    __nv_bfloat16* to[kMoves];
#pragma unroll
    for (int i = 0; i < kMoves; ++i) {
      const int2 mv = s_move[warp][min(i0 + i, count - 1)];
      const __nv_bfloat16* x = row(mv.x);
      to[i] = row(mv.y);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        v[i][2 * p] = *reinterpret_cast<const uint4*>(x + 256 * p);
        v[i][2 * p + 1] = *reinterpret_cast<const uint4*>(x + a.pool.stride_kv + 256 * p);
      }
    }
#pragma unroll
    for (int i = 0; i < kMoves; ++i) {
      if (i0 + i < count) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          *reinterpret_cast<uint4*>(to[i] + 256 * p) = v[i][2 * p];
          *reinterpret_cast<uint4*>(to[i] + a.pool.stride_kv + 256 * p) = v[i][2 * p + 1];
        }
      }
    }
  }
}

template <int KPT, bool CL, bool V4>
cudaError_t launch_select4(const EvictArgs& a, int32_t segs, int32_t ranks, cudaStream_t stream) {
  constexpr int smem = kSelThreads * KPT / 2 * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * ranks), 1, 1);
  cfg.blockDim = dim3(kSelThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel<KPT, CL, V4>, a, ranks);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

template <int KPT, bool CL>
cudaError_t launch_select(const EvictArgs& a, int32_t segs, int32_t ranks, cudaStream_t stream) {
  // four slots a load: pages of whole groups, arrays on 16-byte boundaries (every layer's too)
  const bool v4 = a.pool.page_size % 4 == 0 && ((uintptr_t)a.stats.mass & 15u) == 0 &&
                  ((uintptr_t)a.stats.pos & 15u) == 0;
  return v4 ? launch_select4<KPT, CL, true>(a, segs, ranks, stream)
            : launch_select4<KPT, CL, false>(a, segs, ranks, stream);
}

}  // namespace

// Blocks of the select kernel per segment of up to max_keys keys (1 to 8; the long form has one).
int32_t evict_select_ranks(int32_t max_keys) {
  constexpr int32_t kCta = kSelThreads * 32;
  for (int32_t ranks = 1; ranks <= kMaxCluster; ranks *= 2)
    if (max_keys <= kCta * ranks) return ranks;
  return 1;
}

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t stream) {
  const int32_t segs = a.num_layers * a.plan.num_req * a.pool.num_kv_heads;
  if (segs == 0) return cudaSuccess;
  const int32_t n = a.max_keys, ranks = evict_select_ranks(n);
  // the fewest registers that hold the longest segment: more CTAs share an SM
  if (n <= kSelThreads * 4) return launch_select<4, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 8) return launch_select<8, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 16) return launch_select<16, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 32) return launch_select<32, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 32 * kMaxCluster) return launch_select<32, true>(a, segs, ranks, stream);
  evict_select_long_kernel<<<(unsigned)segs, kLongThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

// A divisor d >= 2 of numbers below 2^31 as multiplier and shift: with 2^(l-1) < d <= 2^l and
// m = ceil(2^(31+l) / d) < 2^32, n / d = (n m) >> (31 + l), as n (m d - 2^(31+l)) < 2^(31+l).
void set_page_divisor(EvictArgs* a) {
  const uint32_t d = (uint32_t)a->pool.page_size;
  a->page_mul = 0;
  a->page_shift = 0;
  if (d < 2) return;
  uint32_t l = 1;
  while ((1ull << l) < d) ++l;
  a->page_mul = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
  a->page_shift = l - 1;
}

int32_t evict_apply_blocks(int32_t keep) { return (keep + kApplySlots - 1) / kApplySlots; }

cudaError_t launch_evict_apply(const EvictArgs& a, cudaStream_t stream) {
  const int32_t segs = a.num_layers * a.plan.num_req * a.pool.num_kv_heads;
  // slots of the budget that no request fills hold -1: they need no block
  const int32_t blocks = evict_apply_blocks(a.max_keys < a.budget ? a.max_keys : a.budget);
  if (segs == 0 || blocks == 0) return cudaSuccess;
  if (a.pool.head_dim == 256)
    evict_apply_kernel<256><<<(unsigned)(segs * blocks), kApplyThreads, 0, stream>>>(a, blocks);
  else
    evict_apply_kernel<512><<<(unsigned)(segs * blocks), kApplyThreads, 0, stream>>>(a, blocks);
  count_launch();
  return cudaGetLastError();
}

}  // namespace pg
