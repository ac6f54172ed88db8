// Eviction from a paged cache by accumulated attention weight ("feat(gemma4): paged KV serving
// across both attention families", Description: one pool per family, pages shared by every layer
// of it, so every layer and head of a request keeps the same number of keys).
//
// A segment is one (layer, request, KV head); its n keys sit in slots [0, n) of the request's
// page list. It keeps n' = min(n, budget): the keys whose position is below num_sink or among
// the last num_recent first, then the largest masses, equal masses by lower slot.
//
//   select  finds the n'-th largest key by counts over the masses' order-preserving bit
//           patterns and writes, for each slot below n', the slot whose key will
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

// Both kernels are launched programmatically: they start, and read the plan (written by copies alone,
// which no programmatic launch overtakes), while the stream's previous kernel ends. Every thread
// waits for that kernel before anything else, also where it then has nothing to do: a kernel that
// could end before the one it waits for would let the next one start too early.
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ select
// One CTA (or a cluster of up to 8) per segment, its keys in registers: thread t of the segment
// holds slots [k t, k (t + 1)), k <= KPT the segment's share of them in groups of four, so slot
// order is thread order and every rank below is a bit count over the thread's 32-bit masks and one
// scan over the threads. Statistics are read in slot order, four slots a load where the pages and
// the arrays allow it (V4), and reach the threads' shares through shared memory (read by their own
// threads, a warp's loads fell into 32 lines: 66 against 47 us on 512 segments of 16,384 keys, with
// the next paragraph's sample).
//
// The keep-th largest order value is searched for in a shrinking range [lo, last], one count over
// the segment per step (compares in registers, a warp reduction and one barrier: no histogram, so
// equal exponents cost nothing). One CTA starts from a range that 128 of its keys suggest, two
// standard deviations of a rank to either side, verified by one double count; it usually holds
// about a sixth of the keys. Then the range is cut in proportion to the counts, every fourth time
// in half; a count that told no keys of it apart shrinks it to the least and the largest key in it,
// so equal keys at the cut end the search (216 segments of up to 667 keys with zeros and equal masses
// 14.0 -> 8.7 us). Once 1024 keys or fewer are in it, they are gathered and only they are counted. The
// search ends when exactly keep keys reach lo (then nothing ties) or the range is one value.
//
// (Keys left in shared memory, with 40 registers a thread and three CTAs of 512 on an SM, were slower: 512
// segments of 8000 keys 36 against 25 us, of 16,384 49 against 47.)
//
// Bound: latency, some 6.5 us of a 16,384-key segment's 14 before the keys are in registers on
// an idle GPU; a segment is read once (8 bytes a key). 512 segments of 8000 keys take 25 us (1.6 TB/s),
// of 16,384 47 us.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;  // at most
constexpr int kMaxCluster = 8;
constexpr int kSampleRanks = 11;  // two standard deviations of a rank in 128 samples

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
template <int NW, bool CL>
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
    int32_t t = __reduce_add_sync(0xffffffffu, lane < NW ? warp_sum[phase][lane] : 0);
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
    const uint32_t w = lane < NW ? (uint32_t)warp_sum[phase][lane] : 0u;
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

// A segment of any length in one CTA, whose keys are read again for each of four 8-bit histogram passes
// and the two ranking passes.
constexpr int kLongThreads = 1024;
struct LongShared {
  uint32_t hist[256];
  int32_t warp_sum[kLongThreads / 32];
  uint32_t prefix;
  int32_t need;
};
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
template <int NT>
__device__ __forceinline__ int32_t block_rank(bool v, int32_t* warp_sum, int32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t b = __ballot_sync(0xffffffffu, v);
  if (lane == 0) warp_sum[warp] = __popc(b);
  __syncthreads();
  int32_t before = 0, all = 0;
  for (int w = 0; w < NT / 32; ++w) {
    const int32_t c = warp_sum[w];
    before += w < warp ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + __popc(b & ((2u << lane) - 1u));
}

// (Not inlined: the select kernel takes it for a plan that grew past its captured launch, and should
// keep its registers for the others.)
template <int NT>
__device__ __noinline__ void select_long(const EvictArgs& a, const Seg& q, int64_t recent, int32_t* src,
                                         LongShared& sh) {
  const int tid = threadIdx.x;
  for (int32_t s = q.keep + tid; s < a.budget; s += NT) src[s] = -1;
  if (q.keep == q.n) {
    for (int32_t s = tid; s < q.keep; s += NT) src[s] = s;
    return;
  }
  // ---- the order value of the keep-th key, and how many of its equals are kept
  uint32_t prefix = 0u;
  int32_t need = q.keep;  // keys still to take among those matching the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += NT) sh.hist[i] = 0u;
    __syncthreads();
    for (int32_t s = tid; s < q.n; s += NT) {
      const uint32_t o = order_at(a, q, recent, s);
      if (shift == 24 || (o >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&sh.hist[(o >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      int32_t left = need;
      int b = 255;
      while (b > 0 && (int32_t)sh.hist[b] < left) left -= (int32_t)sh.hist[b--];
      sh.prefix = prefix | ((uint32_t)b << shift);
      sh.need = left;
    }
    __syncthreads();
    prefix = sh.prefix;
    need = sh.need;
    __syncthreads();
  }
  // ---- kept keys at or past the new length, in slot order, listed in src[0, movers)
  int32_t ties = 0, ties_low = 0, movers = 0;
  for (int32_t s0 = 0; s0 < q.n; s0 += NT) {
    const int32_t s = s0 + tid;
    const uint32_t o = s < q.n ? order_at(a, q, recent, s) : 0u;
    const bool tie = s < q.n && o == prefix;
    int32_t total;
    const int32_t t = block_rank<NT>(tie, sh.warp_sum, &total);
    const bool kept = s < q.n && (o > prefix || (tie && ties + t <= need));
    ties += total;
    ties_low += __syncthreads_count(tie && s < q.keep);
    const bool mover = kept && s >= q.keep;
    const int32_t k = block_rank<NT>(mover, sh.warp_sum, &total);
    if (mover) src[movers + k - 1] = s;
    movers += total;
  }
  __syncthreads();
  // ---- holes below the new length, from the last block of slots to the first: a block reads
  // the list entries of its holes (a hole's rank is at most its slot) before it writes its slots
  int32_t holes_left = movers, ties_left = ties_low;
  for (int32_t s0 = (q.keep - 1) / NT * NT; s0 >= 0; s0 -= NT) {
    const int32_t s = s0 + tid;
    const bool in = s < q.keep;
    const uint32_t o = in ? order_at(a, q, recent, s) : 0u;
    const bool tie = in && o == prefix;
    int32_t total;
    const int32_t t = block_rank<NT>(tie, sh.warp_sum, &total);
    ties_left -= total;
    const bool hole = in && !(o > prefix || (tie && ties_left + t <= need));
    const int32_t k = block_rank<NT>(hole, sh.warp_sum, &total);
    holes_left -= total;
    const int32_t from = hole ? src[holes_left + k - 1] : s;
    __syncthreads();
    if (in) src[s] = from;
    __syncthreads();
  }
}

template <int NT, int KPT, bool CL, bool V4>
__global__ void __launch_bounds__(NT, 1024 / NT) evict_select_kernel(EvictArgs a, int32_t ranks) {
  // kept keys past the new length, by rank: at most half of the cluster's slots, spread over it
  constexpr int kList = NT * KPT / 2;
  constexpr int kGather = NT * KPT < 1024 ? NT * KPT : 1024;  // keys gathered out of the segment
  __shared__ int32_t warp_sum[2][kSelWarps];
  __shared__ int2 cta_sum[2][kMaxCluster];
  __shared__ uint32_t pick[2];
  extern __shared__ uint4 stage[];
  int32_t* const list = reinterpret_cast<int32_t*>(stage);  // (once the keys are in registers)
  const int32_t rank = CL ? (int32_t)(blockIdx.x % ranks) : 0;
  const int32_t seg = CL ? (int32_t)(blockIdx.x / ranks) : (int32_t)blockIdx.x;
  const Seg q = load_seg(a, seg);
  const int64_t recent = recent_from(a, q);
  wait_previous();
  int32_t* src = a.src + (int64_t)seg * a.budget;
  const int tid = threadIdx.x;
  const int32_t step = CL ? NT * ranks : NT, first = rank * NT + tid;
  if (q.keep != q.n && q.n > NT * KPT * (CL ? ranks : 1)) {  // a plan that grew past its captured launch
    static_assert(NT * (KPT / 4 | 1) * 16 >= (int)sizeof(LongShared), "shared memory");
    if (rank == 0) select_long<NT>(a, q, recent, src, *reinterpret_cast<LongShared*>(stage));
    return;
  }
  // every slot keeps its key until a hole below says otherwise
  if (!CL || q.keep == q.n)  // (a cluster that goes on does it below)
    for (int32_t s = first; s < a.budget; s += step) src[s] = s < q.keep ? s : -1;
  if (q.keep == q.n) return;  // (the whole cluster)
  if constexpr (CL) {
    // (the cluster's barriers order every slot before the holes); and every peer runs before its
    // shared memory is written
    for (int32_t s = first; s < a.budget; s += step) src[s] = s < q.keep ? s : -1;
    cluster_barrier();
  }
  // the segment's slots in equal shares: groups of four (whole groups keep V4's vectors in a page)
  const int32_t threads = NT * (CL ? ranks : 1);
  const int32_t share = ((q.n + threads - 1) / threads + 3) & ~3;
  const int32_t s0 = (rank * NT + tid) * share;
  const int32_t s_end = min(q.n, s0 + share);
  // read in the order of the slots, through shared memory to the threads' shares (rows of share / 4
  // groups at an odd pitch, so rows read side by side fall on different banks)
  const int32_t groups = share / 4, pitch = groups | 1;
  {
    const uint32_t mul = (65536u + (uint32_t)groups - 1u) / (uint32_t)groups;  // exact below 8192 groups
    const int32_t c0 = rank * NT * share;
    constexpr int B = KPT < 16 ? KPT / 4 : 4;  // groups of a thread whose loads are in flight
    int32_t page[KPT / 4];                     // (V4) of each group; -2: none
    if constexpr (V4) {
#pragma unroll
      for (int i = 0; i < KPT / 4; ++i) {
        const int32_t s = c0 + 4 * (tid + i * NT);
        page[i] = i < groups && s < q.n ? page_of(a, q, s) : -2;
      }
    }
#pragma unroll
    for (int i0 = 0; i0 < KPT / 4; i0 += B) {
      uint4 k[B];
      if constexpr (V4) {
        int4 pos[B];
        float4 m[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
          pos[i] = make_int4(0, 0, 0, 0);
          m[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (page[i0 + i] >= 0) {
            const int64_t at = stat_at(a, q, page[i0 + i], c0 + 4 * (tid + (i0 + i) * NT));
            pos[i] = *reinterpret_cast<const int4*>(a.stats.pos + at);
            m[i] = *reinterpret_cast<const float4*>(a.stats.mass + at);
          }
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int32_t left = q.n - (c0 + 4 * (tid + (i0 + i) * NT));
          const bool bad = page[i0 + i] < 0;
          k[i].x = left <= 0 ? 0u : bad ? 1u : order_of(a, recent, pos[i].x, m[i].x);
          k[i].y = left <= 1 ? 0u : bad ? 1u : order_of(a, recent, pos[i].y, m[i].y);
          k[i].z = left <= 2 ? 0u : bad ? 1u : order_of(a, recent, pos[i].z, m[i].z);
          k[i].w = left <= 3 ? 0u : bad ? 1u : order_of(a, recent, pos[i].w, m[i].w);
          if (page[i0 + i] == -1) atomicOr(a.status, kStatusBounds);
        }
      } else {
#pragma unroll
        for (int i = 0; i < B; ++i) {
          uint32_t e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t s = c0 + 4 * (tid + (i0 + i) * NT) + e;
            const int32_t page = i0 + i < groups && s < q.n ? page_of(a, q, s) : -2;
            e4[e] = page == -2 ? 0u : 1u;
            if (page >= 0) {
              const int64_t at = stat_at(a, q, page, s);
              e4[e] = order_of(a, recent, a.stats.pos[at], a.stats.mass[at]);
            } else if (page == -1) {
              atomicOr(a.status, kStatusBounds);
            }
          }
          k[i] = make_uint4(e4[0], e4[1], e4[2], e4[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int32_t j = tid + (i0 + i) * NT, t = (int32_t)((uint32_t)j * mul >> 16);
        if (i0 + i < groups) stage[t * pitch + j - t * groups] = k[i];
      }
    }
  }
  __syncthreads();
  uint32_t key[KPT];
#pragma unroll
  for (int i = 0; i < KPT / 4; ++i) {
    const uint4 k = i < groups ? stage[tid * pitch + i] : make_uint4(0u, 0u, 0u, 0u);
    key[4 * i] = k.x;
    key[4 * i + 1] = k.y;
    key[4 * i + 2] = k.z;
    key[4 * i + 3] = k.w;
  }
  Counter<NT / 32, CL> count{warp_sum, cta_sum, rank, ranks, 0};
  // ---- the keep-th largest order value: it lies in [lo, last], reach keys are lo or more and above
  // (fewer than keep) are more than last
  uint32_t lo = 1u, last = 0xFFFFFFFFu;
  int32_t reach = q.n, above = 0;
  auto at_least = [&](uint32_t v) {
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < KPT; i += 4) {
      if (i < share)  // (uniform)
        c += (key[i] >= v ? 1 : 0) + (key[i + 1] >= v ? 1 : 0) + (key[i + 2] >= v ? 1 : 0) +
             (key[i + 3] >= v ? 1 : 0);
    }
    return c;
  };
  if constexpr (!CL) {
    // two values around it, by the ranks of a sample: 128 threads' first keys
    constexpr int kEach = NT / 128, kPart = 128 / kEach;  // threads to a sample, keys that each looks at
    __shared__ uint4 sample[kEach][kPart / 4 + 1];        // (the parts a group apart)
    const int i = tid / kEach, part = tid % kEach;
    uint32_t* const slot = reinterpret_cast<uint32_t*>(sample[i / kPart]) + i % kPart;
    if (part == 0) *slot = key[0];
    if (tid < 2) pick[tid] = 1u;
    __syncthreads();
    const uint32_t own = *slot;
    int32_t c1 = 0;  // of the sample, keys not below this one
#pragma unroll
    for (int g = 0; g < kPart / 4; ++g) {
      const uint4 k = sample[part][g];
      c1 += (k.x >= own ? 1 : 0) + (k.y >= own ? 1 : 0) + (k.z >= own ? 1 : 0) + (k.w >= own ? 1 : 0);
    }
#pragma unroll
    for (int o = 1; o < kEach; o <<= 1) c1 += __shfl_xor_sync(0xffffffffu, c1, o);
    const int32_t held = ((q.n + share - 1) / share + kEach - 1) / kEach;  // sampled threads that hold keys
    const int32_t r = q.keep * held / q.n;
    const uint32_t mx = __reduce_max_sync(0xffffffffu, c1 >= r + kSampleRanks ? own : 0u);
    const uint32_t my = __reduce_max_sync(0xffffffffu, c1 >= r - kSampleRanks ? own : 0u);
    if ((tid & 31) == 0) {
      atomicMax(&pick[0], mx);
      atomicMax(&pick[1], my);
    }
    __syncthreads();
    const uint32_t x = pick[0];
    const bool top = pick[1] == 0xFFFFFFFFu || r - kSampleRanks <= 0;  // nothing is known past it
    const uint32_t y = top ? 0u : pick[1] + 1u;
    // (at most 16,384 keys: two counts of 16 bits)
    const uint32_t c = (uint32_t)count.total(at_least(x) + (top ? 0 : at_least(y) << 16));
    const int32_t cx = (int32_t)(c & 0xFFFFu), cy = (int32_t)(c >> 16);
    if (cx >= q.keep) {
      lo = x;
      reach = cx;
    } else {
      last = x - 1u;
      above = cx;
    }
    if (!top && cx >= q.keep) {
      if (cy >= q.keep) {
        lo = y;
        reach = cy;
      } else {
        last = y - 1u;
        above = cy;
      }
    }
  }
  int32_t tries = 0;
  bool moved = true;  // the last count told keys of the range apart
  auto middle = [&]() {  // in (lo, last]
    const uint32_t span = last - lo;
    ++tries;
    if (span > (1u << 25) || !moved || (tries & 3) == 0) return lo + (span >> 1) + 1u;
    const float f = (float)(reach - q.keep) / (float)(reach - above);
    return lo + max(1u, min(span, (uint32_t)((float)span * f)));
  };
  auto narrow = [&](uint32_t v, int32_t c) {
    moved = c != reach && c != above;
    if (c >= q.keep) {
      lo = v;
      reach = c;
    } else {
      last = v - 1u;
      above = c;
    }
  };
  // equal keys at the cut: the range shrinks to the least and largest key in it (one CTA; a cluster
  // goes on by halves)
  auto tighten = [&](uint32_t least, uint32_t most) {
    if (tid < 2) pick[tid] = tid == 0 ? 0xFFFFFFFFu : 0u;
    __syncthreads();
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if ((tid & 31) == 0) {
      atomicMin(&pick[0], least);
      atomicMax(&pick[1], most);
    }
    __syncthreads();
    lo = pick[0];
    last = pick[1];
    moved = true;
  };
  while (lo < last && reach != q.keep && (CL || reach - above > kGather)) {
    if (!CL && !moved) {
      uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
      for (int i = 0; i < KPT; ++i) {
        const bool in = key[i] >= lo && key[i] <= last;
        least = in ? min(least, key[i]) : least;
        most = in ? max(most, key[i]) : most;
      }
      tighten(least, most);
      continue;
    }
    const uint32_t v = middle();
    narrow(v, count.total(at_least(v)));
  }
  if constexpr (!CL) {
    if (lo < last && reach != q.keep) {
      // the few keys of the range
      int32_t mine = 0;
#pragma unroll
      for (int i = 0; i < KPT; ++i) mine += key[i] >= lo && key[i] <= last ? 1 : 0;
      int2 all;
      int32_t at = count.before(mine, 0, &all).x;
#pragma unroll
      for (int i = 0; i < KPT; ++i)
        if (key[i] >= lo && key[i] <= last) list[at++] = (int32_t)key[i];
      __syncthreads();
      const int32_t past = above;  // keys past the range
      uint32_t few[kGather / NT];
#pragma unroll
      for (int i = 0; i < kGather / NT; ++i) {
        const int32_t x = tid + i * NT;
        few[i] = x < all.x ? (uint32_t)list[x] : 0u;
      }
      while (lo < last && reach != q.keep) {
        if (!moved) {
          uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
          for (int i = 0; i < kGather / NT; ++i) {
            const bool in = few[i] >= lo && few[i] <= last;
            least = in ? min(least, few[i]) : least;
            most = in ? max(most, few[i]) : most;
          }
          tighten(least, most);
          continue;
        }
        const uint32_t v = middle();
        int32_t c = past;
#pragma unroll
        for (int i = 0; i < kGather / NT; ++i) c += __syncthreads_count(few[i] >= v);
        narrow(v, c);
      }
    }
  }
  const uint32_t cut = lo;
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

// Segments longer than a cluster's registers (131,072 keys): one of 140,000 keys takes 1.06 ms, 16 of
// 200,000 1.58 ms (the longest of the form above, 131,072 keys, 37 us).
__global__ void __launch_bounds__(kLongThreads) evict_select_long_kernel(EvictArgs a) {
  __shared__ LongShared sh;
  const Seg q = load_seg(a, (int32_t)blockIdx.x);
  select_long<kLongThreads>(a, q, recent_from(a, q), a.src + (int64_t)blockIdx.x * a.budget, sh);
}

// ------------------------------------------------------------------ apply
// A warp takes S kept slots of one segment (up to 32, or a multiple of 32: S / 32 a lane): it lists
// the slots whose key comes from elsewhere, then moves them four at a time, each row's 16-byte pieces
// spread over the lanes (at head_dim 512 a lane has 16 loads in flight), so the moves of a warp
// wait for memory once per four. Bound: 4 D bytes read and written per move, and the map read.
constexpr int kApplyThreads = 256, kApplyWarps = kApplyThreads / 32, kMoves = 4;
constexpr int kApplyDense = 16, kApplySparse = 256;  // slots of a warp (see launch_evict_apply)
template <int D, int S>
__global__ void __launch_bounds__(kApplyThreads) evict_apply_kernel(EvictArgs a, int32_t blocks_per_seg) {
  constexpr int N = S < 32 ? 1 : S / 32;
  __shared__ int2 s_move[kApplyWarps][S];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t seg = (int32_t)blockIdx.x / blocks_per_seg;
  const int32_t t0 = ((int32_t)blockIdx.x % blocks_per_seg) * (kApplyWarps * S) + warp * S + lane;
  const int32_t* src = a.src + (int64_t)seg * a.budget;
  const Seg q = load_seg(a, seg);
  wait_previous();
  int32_t from[N];
#pragma unroll
  for (int i = 0; i < N; ++i) from[i] = (S >= 32 || lane < S) && t0 + 32 * i < a.budget ? src[t0 + 32 * i] : -1;
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; ++i) any |= from[i] >= 0 && from[i] != t0 + 32 * i;
  if (!__any_sync(0xffffffffu, any)) return;
  // rows (page * page_size + offset) of each move, listed by the warp
  int32_t count = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
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

template <int NT, int KPT, bool CL, bool V4>
cudaError_t launch_select4(const EvictArgs& a, int32_t segs, int32_t ranks, cudaStream_t stream) {
  constexpr int smem = NT * (KPT / 4 | 1) * 16;  // (the list: NT KPT / 2 numbers)
  static PerDeviceOnce setup;
  int dev = 0, unused = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = setup.get(dev, [](int*) {
    return cudaFuncSetAttribute(evict_select_kernel<NT, KPT, CL, V4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem);
  }, &unused);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * ranks), 1, 1);
  cfg.blockDim = dim3(NT, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel<NT, KPT, CL, V4>, a, ranks);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

template <int NT, int KPT, bool CL>
cudaError_t launch_select(const EvictArgs& a, int32_t segs, int32_t ranks, cudaStream_t stream) {
  // four slots a load: pages of whole groups, arrays on 16-byte boundaries (every layer's too)
  const bool v4 = a.pool.page_size % 4 == 0 && ((uintptr_t)a.stats.mass & 15u) == 0 &&
                  ((uintptr_t)a.stats.pos & 15u) == 0;
  return v4 ? launch_select4<NT, KPT, CL, true>(a, segs, ranks, stream)
            : launch_select4<NT, KPT, CL, false>(a, segs, ranks, stream);
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
  // the fewest registers that hold the longest segment
  static PerDeviceOnce device;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = device.get(dev, [dev](int* v) { return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev); }, &sms);
  if (e != cudaSuccess) return e;
  // Two CTAs of 512 threads fill an SM's registers. Where there are more segments than that, 256
  // threads each: four of their chains of loads and counts then overlap on an SM (512 segments of
  // 2048, 4096, 8000 keys: 12.8, 15.4, 25 against 15.3, 19.7, 30 us).
  // Short segments need fewer threads, and the barriers among fewer are shorter: 240 segments of 300
  // keys take 6.8 us in 128 threads against 9.5 in 512, 1000 of 1000 keys 14.2 in 256 against 24.8.
  if (n <= 128 * 4) return launch_select<128, 4, false>(a, segs, 1, stream);
  if (n <= 256 * 4) return launch_select<256, 4, false>(a, segs, 1, stream);
  if (segs > 2 * sms) {
    if (n <= 256 * 8) return launch_select<256, 8, false>(a, segs, 1, stream);
    if (n <= 256 * 16) return launch_select<256, 16, false>(a, segs, 1, stream);
    if (n <= 256 * 32) return launch_select<256, 32, false>(a, segs, 1, stream);
  }
  if (n <= kSelThreads * 4) return launch_select<kSelThreads, 4, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 8) return launch_select<kSelThreads, 8, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 16) return launch_select<kSelThreads, 16, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 32) return launch_select<kSelThreads, 32, false>(a, segs, 1, stream);
  if (n <= kSelThreads * 32 * kMaxCluster) return launch_select<kSelThreads, 32, true>(a, segs, ranks, stream);
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

// At most as many blocks of the apply kernel per segment of `keep` kept slots.
int32_t evict_apply_blocks(int32_t keep) { return (keep + kApplyWarps * kApplyDense - 1) / (kApplyWarps * kApplyDense); }

cudaError_t launch_evict_apply(const EvictArgs& a, cudaStream_t stream) {
  const int32_t segs = a.num_layers * a.plan.num_req * a.pool.num_kv_heads;
  const int32_t slots = a.slots;
  if (segs == 0 || slots == 0) return cudaSuccess;
  static PerDeviceOnce device;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  err = device.get(dev, [dev](int* v) { return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev); }, &sms);
  if (err != cudaSuccess) return err;
  // Few slots a warp keep its chain of moves short: half of 64 segments of 16,384 keys moved in 170 us
  // against 182 with 128 slots, two thirds of 192 segments of 321 in 18 against 42. Where next to none
  // move (a request gives up at most max_keys - budget keys as the plan stands) and there are more such blocks than fit
  // the GPU at once, reading the map is all there is to do, and that wants many slots: one moved key
  // in each of 512 segments of 4096 took 33 us with 16 slots, 7.8 with 128 and 5.7 with 256.
  int32_t blocks = evict_apply_blocks(slots);
  const bool sparse = (int64_t)(a.max_keys - slots) * 32 <= slots && segs * blocks > 8 * sms;
  if (sparse) blocks = (slots + kApplyWarps * kApplySparse - 1) / (kApplyWarps * kApplySparse);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(segs * blocks), 1, 1);
  cfg.blockDim = dim3(kApplyThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, a, blocks); };
  const cudaError_t e =
      a.pool.head_dim == 256
          ? (sparse ? run(evict_apply_kernel<256, kApplySparse>) : run(evict_apply_kernel<256, kApplyDense>))
          : (sparse ? run(evict_apply_kernel<512, kApplySparse>) : run(evict_apply_kernel<512, kApplyDense>));
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace pg
