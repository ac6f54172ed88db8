// Accumulated attention weights of a prefill step on the tensor cores (tcgen05 + TMEM + TMA): the
// second pass behind the attention (attn_mass.cu says what is summed). Page sizes 8, 16, 32, ...
//
// S^T = K Q^T with keys as MMA rows: a key is a TMEM lane, so its sum over query rows runs along
// one thread's own columns, in registers, in one fixed order and without atomics.
//
// A segment is (request, KV head, 256 keys) with the query tiles (256 rows) that see some of its
// keys; the segments in order give the step's T tiles, and cluster s of S (one per SM pair,
// persistent) takes tiles [s T / S, (s + 1) T / S): equal work to one tile whatever the lengths,
// the causal triangle included, and few K loads. MMAs run in the 2-SM form (M = 256 keys, N = 256
// query rows, K = 16). CTA c keeps its 128 keys of K in two 64 KB part slots (256 d each: head_dim
// 512 fills both, head_dim 256 loads the next segment's K into the other) and streams its half
// (128 rows) of every query tile through a ring of 16 KB stages (128 rows x 64 d). Two 256-column
// score buffers fill TMEM, so the sums of one tile overlap the products of the next. A query byte
// is used for 256 keys: at the full MMA rate the rings take 32 bytes a clock and SM from L2; with
// 128 keys they would ask for 64, which L2 does not give all SMs at once.
//
//   warp 0     producer: a segment's K parts (one 4-D box per page), each just before the query
//              stages that need it, and the query tiles
//   warp 1     MMA issuer (leader CTA)
//   warps 2-9  sums: two warps per TMEM lane quarter, 128 columns each; exp2(s c - lse) on fp32
//              pairs, masked on boundary tiles only. A tile's 128 terms are summed in four
//              accumulators and then added to the segment's sum with a compensated addition.
//
// A segment inside one cluster's range updates the statistics at its end; one that is cut leaves
// a record of 256 sums per cluster, and the join kernel adds a segment's records in order. Cuts
// follow from the plan alone, so equal calls give equal bits. Every role finds its own place in
// the order (a scan over the requests and one over the key tiles of one request).
//
// Every wait is bounded (a wait that runs out sets the device status word and the CTA leaves).
#include "bounded.cuh"
#include "mass.cuh"
#include "pg_internal.h"
#include "tc_ptx.cuh"

#include <algorithm>

namespace pg {
namespace {

constexpr int kMK = 128;          // keys per CTA
constexpr int kNQ = 256;          // query rows per tile (both CTAs' halves)
constexpr int kStage = 16 * 1024; // 128 query rows x 64 d
constexpr int kThreadsMass = 320;
constexpr int kMaxClusters = 128;

template <int D>
struct MassCfg {
  static constexpr int KP = D / 256;             // 256-d parts of a key row
  static constexpr int CH = D / 64;              // ring stages per query tile
  static constexpr int NS = 5;                   // ring stages
  static constexpr int PART = kMK * 512;         // one K part slot
  static constexpr int OFF_Q = 2 * PART;
  static constexpr int OFF_LSE = OFF_Q + NS * kStage;      // [2 tile parities][256] -lse, log2 units
  static constexpr int OFF_X = OFF_LSE + 2 * kNQ * 4;      // [2 segment parities][2 halves][128] sums
  static constexpr int OFF_BAR = OFF_X + 4 * kMK * 4;
  // FULL[NS], EMPTY[NS], KFULL[2], KEMPTY[2], AFULL[2], AEMPTY[2], LSE[2 halves][2 parities],
  // PAIR[4], DRAIN
  static constexpr int NBAR = 2 * NS + 4 + 4 + 4 + 4 + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A place in the order of segments, and the tiles [t, t_hi) that this cluster takes of the current
// one. Every lane of every warp that walks the order holds the same values.
struct SegWalk {
  MassReq q;
  MassTiles mt;
  int32_t r, g, kt, key_tiles;
  int32_t t, t_hi;
  int64_t left;  // the cluster's tiles from here on, this segment's included
  bool first;    // nothing of this cluster before it
  bool cut;      // the segment also has tiles in another cluster
};
__device__ __forceinline__ int64_t request_tiles(const AttnArgs& a, int32_t r, MassReq* q) {
  *q = mass_req(a.plan, r, a.pool.page_size);
  const int32_t kts = (q->n + 2 * kMK - 1) / (2 * kMK);
  int64_t n = 0;
  for (int32_t k = 0; k < kts; ++k) {
    const MassTiles t = mass_tiles(a, *q, k);
    n += t.end - t.first;
  }
  return n;
}
__device__ __forceinline__ void take(SegWalk& w) {
  const int64_t n = min((int64_t)(w.mt.end - w.t), w.left);
  w.t_hi = w.t + (int32_t)n;
  w.cut = w.t > w.mt.first || w.t_hi < w.mt.end;
}
// The cluster's first segment; left 0 when it has none. *total: tiles of the step.
__device__ __forceinline__ SegWalk walk_start(const AttnArgs& a, int32_t s, int32_t S, int64_t* total) {
  const int32_t R = a.plan.num_req, Hkv = a.pool.num_kv_heads, lane = threadIdx.x & 31;
  SegWalk w;
  MassReq q;
  // tiles per request, a lane each; the first 32 requests' counts are kept for the second scan
  const int64_t held = lane < R ? request_tiles(a, lane, &q) * Hkv : 0;
  auto scan = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  int64_t T = __shfl_sync(0xffffffffu, scan(held), 31);
  for (int32_t c = 32; c < R; c += 32)
    T += __shfl_sync(0xffffffffu, scan(c + lane < R ? request_tiles(a, c + lane, &q) * Hkv : 0), 31);
  *total = T;
  const int64_t u0 = s * T / S, u1 = (s + 1) * T / S;
  w.left = u1 - u0;
  if (w.left == 0) return w;
  int64_t run = 0, in_req = 0;
  w.r = 0;
  for (int32_t c = 0; c < R; c += 32) {
    const int64_t v = c == 0 ? held : c + lane < R ? request_tiles(a, c + lane, &q) * Hkv : 0;
    const int64_t incl = scan(v);
    const uint32_t past = __ballot_sync(0xffffffffu, run + incl > u0);
    if (past) {
      const int f = __ffs(past) - 1;
      w.r = c + f;
      in_req = u0 - run - __shfl_sync(0xffffffffu, incl - v, f);
      break;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  const int64_t per_head = request_tiles(a, w.r, &w.q);
  w.g = (int32_t)(in_req / per_head);
  int64_t at = in_req % per_head;
  w.key_tiles = (w.q.n + 2 * kMK - 1) / (2 * kMK);
  for (w.kt = 0;; ++w.kt) {
    w.mt = mass_tiles(a, w.q, w.kt);
    if (at < w.mt.end - w.mt.first) break;
    at -= w.mt.end - w.mt.first;
  }
  w.t = w.mt.first + (int32_t)at;
  w.first = true;
  take(w);
  return w;
}
// The next segment with tiles; false when the cluster's range ends.
__device__ __forceinline__ bool walk_next(const AttnArgs& a, SegWalk& w) {
  w.left -= w.t_hi - w.t;
  if (w.left <= 0) return false;
  do {
    if (++w.kt >= w.key_tiles) {
      w.kt = 0;
      if (++w.g == a.pool.num_kv_heads) {
        w.g = 0;
        w.q = mass_req(a.plan, ++w.r, a.pool.page_size);
        w.key_tiles = (w.q.n + 2 * kMK - 1) / (2 * kMK);
      }
    }
    w.mt = mass_tiles(a, w.q, w.kt);
  } while (w.mt.first >= w.mt.end);
  w.t = w.mt.first;
  w.first = false;
  take(w);
  return true;
}

// What the join needs to know of a segment that starts in cluster s and goes on past it.
struct alignas(16) MassCut {
  int32_t r, g, kt, slot;  // slot: its record in cluster s (0: the cluster's first segment, 1)
  int32_t last;            // the last cluster that has tiles of it (-1: no such segment)
  int32_t empty;           // the cluster has no tiles, and no record
  int32_t sparse;          // the step has fewer tiles than clusters: some are empty
  int32_t pad;
};

template <int D>
__global__ void __launch_bounds__(kThreadsMass, 1)
mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               MassArgs m, int32_t box_rows) {
  using C = MassCfg<D>;
  constexpr int NS = C::NS, CH = C::CH, KP = C::KP;
  const AttnArgs& a = m.attn;
  const PlanDev& pl = a.plan;
  const int32_t Hkv = a.pool.num_kv_heads, ps = a.pool.page_size, G = a.group, Hq = a.num_qo_heads;
  const int32_t S = (int32_t)gridDim.x >> 1, s = (int32_t)blockIdx.x >> 1;
  MassCut* const cuts = reinterpret_cast<MassCut*>(m.ws);
  float* const recs = reinterpret_cast<float*>(cuts + kMaxClusters);  // [S][2][256]

  int64_t total;
  SegWalk w = walk_start(a, s, S, &total);

  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::OFF_BAR;
  auto FULL = [&](int x) { return bars + 8u * x; };
  auto EMPTY = [&](int x) { return bars + 8u * (NS + x); };
  const uint32_t KFULL = bars + 8u * (2 * NS), KEMPTY = KFULL + 16, AFULL = KFULL + 32, AEMPTY = KFULL + 48,
                 LSEB = KFULL + 64, PAIR = KFULL + 96, DRAIN = KFULL + 128;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, a.status, a.wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  auto LEAD = [&](uint32_t bar) { return mapa(bar, 0); };

  // the join's launch overlaps this kernel; this one's own start overlaps the attention's tail
  // (programmatic launches): only the sums need what the attention wrote, its lse
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (w.left == 0) {  // (both CTAs of the cluster)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (leader && threadIdx.x == 0) cuts[s] = MassCut{0, 0, 0, 0, -1, 1, 1, 0};
    return;
  }
  if (leader && warp == 2 && lane == 0) cuts[s] = MassCut{0, 0, 0, 0, -1, 0, 0, 0};  // until its end
  if (threadIdx.x == 0) {
    for (int x = 0; x < NS; ++x) {
      mbar_init(FULL(x), 2);  // one arrival (with its byte count) from each CTA's producer
      mbar_init(EMPTY(x), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(KFULL + 8 * b, 2);
      mbar_init(KEMPTY + 8 * b, 1);
      mbar_init(AFULL + 8 * b, 1);
      mbar_init(AEMPTY + 8 * b, 16);  // the sum warps of both CTAs
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(LSEB + 8 * i, 4);  // the four warps of a column half
      mbar_init(PAIR + 8 * i, 2);
    }
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int32_t TQ = kNQ / G;  // tokens per query tile

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true, more = true;
    int32_t kc = 0;  // K parts loaded
    int x = 0, round = 0;
    const int nbox = kMK / box_rows;
    while (ok && more) {
      const int32_t rel0 = w.kt * (2 * kMK) + (int32_t)rank * kMK;
      for (int32_t t = w.t; ok && t < w.t_hi; ++t) {
        const int32_t tok = w.q.q0 + t * TQ + (int32_t)rank * (TQ / 2);
        for (int p = 0; ok && p < KP; ++p) {
          if (t == w.t) {
            // part p of the segment's K, once the part that used its slot has been multiplied; lane
            // l takes page boxes l, l + 32, ...
            const int sl = kc & 1;
            int go = 1;
            if (lane == 0) go = mbar_wait_inline(KEMPTY + 8 * sl, ((kc >> 1) & 1) ^ 1, wc) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, go, 0)) {
              ok = false;
              break;
            }
            uint32_t bytes = 0u;
            bool bad = false;
            for (int b = lane; b < nbox; b += 32) {
              const int32_t rel = rel0 + b * box_rows;
              if (rel >= w.q.n) continue;
              if (mass_page(pl, w.q, rel, ps, a.pool.num_pages) == a.pool.num_pages) bad = true;
              else bytes += (uint32_t)box_rows * 512u;
            }
            bytes = __reduce_add_sync(0xffffffffu, bytes);
            if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kStatusBounds);
            if (lane == 0) mbar_expect_tx_cl_relaxed(LEAD(KFULL + 8 * sl), bytes);
            __syncwarp();
            for (int b = lane; b < nbox; b += 32) {
              const int32_t rel = rel0 + b * box_rows;
              if (rel >= w.q.n) continue;
              const int32_t page = mass_page(pl, w.q, rel, ps, a.pool.num_pages);
              if (page == a.pool.num_pages) continue;
              const int32_t row = (int32_t)(((int64_t)page * 2 * Hkv + w.g) * ps + rel % ps);
              tma_load_4d(base + sl * C::PART + b * box_rows * 512, &tm_k, 0, 0, p * 4, row / 8,
                          LEAD(KFULL + 8 * sl));
            }
            __syncwarp();
            ++kc;
          }
          // four stages of the query tile
          int go = 1;
          if (lane == 0) {
            int y = x, rd = round;
            for (int ch = 4 * p; go && ch < 4 * p + 4; ++ch) {
              if (!mbar_wait_inline(EMPTY(y), (rd & 1) ^ 1, wc)) {
                go = 0;
                break;
              }
              mbar_expect_tx_cl_relaxed(LEAD(FULL(y)), kStage);
              tma_load_3d(base + C::OFF_Q + y * kStage, &tm_q, ch * 64, w.g * G, tok, LEAD(FULL(y)));
              if (++y == NS) { y = 0; ++rd; }
            }
          }
          x += 4;
          if (x >= NS) { x -= NS; ++round; }
          if (!__shfl_sync(0xffffffffu, go, 0)) ok = false;
        }
      }
      more = ok && walk_next(a, w);
    }
    if (!ok) {
      const uint64_t t0 = globaltimer();  // the copies already issued land before the CTA leaves
      while (globaltimer() - t0 < 100000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the leader's)
    constexpr uint32_t IDESC = idesc_bf16(2 * kMK, kNQ, false);
    auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
      const bool y = lane == 0 ? mbar_wait_inline(bar, parity, wc) : false;
      return __shfl_sync(0xffffffffu, y ? 1 : 0, 0) != 0;
    };
    if (leader) {
      bool ok = true, more = true;
      int x = 0, round = 0;
      int32_t i = 0, kc = 0;
      while (ok && more) {
        for (int32_t t = w.t; ok && t < w.t_hi; ++t, ++i) {
          const int b = i & 1;
          ok = wait1(AEMPTY + 8 * b, ((i >> 1) & 1) ^ 1);
          for (int ch = 0; ok && ch < CH; ++ch) {
            const int32_t kp = kc + (ch >> 2);  // this segment's K part, counted from the start
            if (t == w.t && (ch & 3) == 0) ok = wait1(KFULL + 8 * (kp & 1), (kp >> 1) & 1);
            ok = ok && wait1(FULL(x), round & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = sdesc(base + (kp & 1) * C::PART + (ch & 3) * 1024, 16, 4096);
            const uint64_t qd = sdesc(base + C::OFF_Q + x * kStage, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss<IDESC>(tmem + b * kNQ, kd + kk * 2, qd + kk * 2, (ch > 0 || kk > 0) ? 1u : 0u);
            mma_commit(EMPTY(x));
            if (t == w.t_hi - 1 && (ch & 3) == 3) mma_commit(KEMPTY + 8 * (kp & 1));
            if (++x == NS) { x = 0; ++round; }
          }
          if (ok) mma_commit(AFULL + 8 * b);
        }
        kc += KP;
        more = ok && walk_next(a, w);
      }
      mma_commit(DRAIN);
    }
  } else {
    // ------------------------------------------------------------ sums
    const int quarter = warp & 3, h = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;                   // TMEM lane: this thread's key
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + h * (kNQ / 2);
    const int32_t W = a.window_left, sink = a.num_sink;
    const int gsh = __ffs(G) - 1;
    float* const lbuf = reinterpret_cast<float*>(gbase + C::OFF_LSE) + h * (kNQ / 2);
    // -lse (log2 units) of this thread's column of tile t; -inf: not a row of the request
    const int col = h * (kNQ / 2) + row;
    auto fetch = [&](int32_t t) -> float {
      const int32_t tk = t * TQ + (col >> gsh);
      if (tk >= w.q.len) return -INFINITY;
      return a.lse[(int64_t)(w.q.q0 + tk) * Hq + w.g * G + (col & (G - 1))] * -1.4426950408889634f;
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool ok = true, more = true;
    const float2 sc = make_float2(a.sm_scale_log2, a.sm_scale_log2);
    int32_t i = 0;
    for (int32_t seg = 0; ok && more; ++seg) {
      const int32_t rel = w.kt * (2 * kMK) + (int32_t)rank * kMK + row, j = w.q.ks0 + rel;
      const bool kvalid = rel < w.q.n;
      float nxt = fetch(w.t);
      float sum = 0.f, comp = 0.f;
      for (int32_t t = w.t; ok && t < w.t_hi; ++t, ++i) {
        const int b = i & 1;
        // this half's 128 values; the barrier of this parity also shows that all four warps are past
        // tile i - 1, so tile i + 1's values may replace it
        lbuf[b * kNQ + row] = nxt;
        if (t + 1 < w.t_hi) nxt = fetch(t + 1);
        __syncwarp();
        const uint32_t lb = LSEB + 8 * (h * 2 + b);
        if (lane == 0) mbar_arrive(lb);
        if (!__all_sync(0xffffffffu, mbar_wait_inline(lb, (i >> 1) & 1, wc)) ||
            !__all_sync(0xffffffffu, mbar_wait_inline(AFULL + 8 * b, (i >> 1) & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the half's rows: positions p0 .. p1
        const int32_t tk0 = t * TQ + ((h * (kNQ / 2)) >> gsh), ntk = (kNQ / 2) >> gsh;
        const int32_t p0 = w.q.sp + tk0, p1 = p0 + ntk - 1;
        const bool interior = __all_sync(
            0xffffffffu, tk0 + ntk <= w.q.len && kvalid && j <= p0 && (W < 0 || p1 - j <= W || j < sink));
        // this key's columns of the half: tokens from j - sp on, to the window's last (or the last)
        int32_t c_lo = 0, c_hi = 0;
        if (!interior && kvalid) {
          const int64_t t0 = max((int64_t)j - w.q.sp - tk0, (int64_t)0);
          int64_t t1 = min(ntk, w.q.len - tk0);
          if (W >= 0 && j >= sink) t1 = min(t1, (int64_t)j + W - w.q.sp - tk0 + 1);
          c_lo = (int32_t)min(t0, (int64_t)ntk) << gsh;
          c_hi = (int32_t)max(t1, (int64_t)0) << gsh;
        }
        float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float4* lv = reinterpret_cast<const float4*>(lbuf + b * kNQ);
#pragma unroll 1
        for (int cb = 0; cb < kNQ / 2; cb += 64) {
          uint32_t sv[64];
          tmem_ld32(tl + b * kNQ + cb, sv);
          tmem_ld32(tl + b * kNQ + cb + 32, sv + 32);
          tmem_wait_ld();
          if (cb + 64 == kNQ / 2) {
            // every column is read: the buffer is free for the tile after next
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cl(LEAD(AEMPTY + 8 * b));
          }
          if (interior) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float4 l4 = lv[cb / 4 + k];
              const float2 e0 = __ffma2_rn(
                  make_float2(__uint_as_float(sv[4 * k]), __uint_as_float(sv[4 * k + 1])), sc, make_float2(l4.x, l4.y));
              const float2 e1 = __ffma2_rn(
                  make_float2(__uint_as_float(sv[4 * k + 2]), __uint_as_float(sv[4 * k + 3])), sc, make_float2(l4.z, l4.w));
              s2[0] = __fadd2_rn(s2[0], make_float2(ex2(e0.x), ex2(e0.y)));
              s2[1] = __fadd2_rn(s2[1], make_float2(ex2(e1.x), ex2(e1.y)));
            }
          } else {
            // the columns of the rows that see this key, as 64 bits: a test per score
            const uint64_t vis = bits_below(c_hi - cb) & ~bits_below(c_lo - cb);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float4 l4 = lv[cb / 4 + k];
              const float2 e0 = __ffma2_rn(
                  make_float2(__uint_as_float(sv[4 * k]), __uint_as_float(sv[4 * k + 1])), sc, make_float2(l4.x, l4.y));
              const float2 e1 = __ffma2_rn(
                  make_float2(__uint_as_float(sv[4 * k + 2]), __uint_as_float(sv[4 * k + 3])), sc, make_float2(l4.z, l4.w));
              s2[0] = __fadd2_rn(s2[0], make_float2(ex2((vis >> (4 * k)) & 1u ? e0.x : -INFINITY),
                                                    ex2((vis >> (4 * k + 1)) & 1u ? e0.y : -INFINITY)));
              s2[1] = __fadd2_rn(s2[1], make_float2(ex2((vis >> (4 * k + 2)) & 1u ? e1.x : -INFINITY),
                                                    ex2((vis >> (4 * k + 3)) & 1u ? e1.y : -INFINITY)));
            }
          }
        }
        const float part = (s2[0].x + s2[1].x) + (s2[0].y + s2[1].y);
        // compensated: the sum may add many tiles (an infinite or NaN sum stays as it is)
        const float y = part - comp, z = sum + y;
        comp = isfinite(z) ? (z - sum) - y : 0.f;
        sum = z;
      }
      if (!ok) break;
      // the two column halves of a key (buffers by segment parity: the partner has read the one of
      // two segments ago before it arrived for the last one)
      float* const xs = reinterpret_cast<float*>(gbase + C::OFF_X) + (seg & 1) * 2 * kMK;
      xs[h * kMK + row] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(PAIR + 8 * quarter);
      ok = __all_sync(0xffffffffu, mbar_wait(PAIR + 8 * quarter, seg & 1, wc));
      if (ok && h == 0) {
        const float both = xs[row] + xs[kMK + row];
        if (w.cut) {
          recs[((int64_t)s * 2 + (w.first ? 0 : 1)) * (2 * kMK) + rank * kMK + row] = both;
        } else if (kvalid && mass_seen(a, w.q, rel)) {
          const int32_t page = mass_page(pl, w.q, rel, ps, a.pool.num_pages);
          if (page < a.pool.num_pages) mass_store(a, w.q, page, w.g, rel, both);  // (else: reported)
        }
      }
      const bool last = w.left == w.t_hi - w.t;
      if (last && leader && warp == 2 && lane == 0) {
        // a segment that starts here and goes on: its end among the clusters, for the join
        MassCut cut{w.r, w.g, w.kt, w.first ? 0 : 1, -1, 0, total < S ? 1 : 0, 0};
        if (w.t == w.mt.first && w.t_hi < w.mt.end) {
          const int64_t end = (int64_t)(s + 1) * total / S + (w.mt.end - w.t_hi);  // its tiles end here
          cut.last = (int32_t)((end * S - 1) / total);
        }
        cuts[s] = cut;
      }
      more = walk_next(a, w);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1 && lane == 0) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(DRAIN, 0)) {
      if (globaltimer() - t0 > a.wait_ns) {
        atomicOr(a.status, kStatusTimeout);
        break;
      }
    }
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Block s: the segment that starts in cluster s and goes on past it, a thread per key.
__global__ void __launch_bounds__(2 * kMK) mass_join_kernel(MassArgs m) {
  const AttnArgs& a = m.attn;
  const MassCut* cuts = reinterpret_cast<const MassCut*>(m.ws);
  const float* recs = reinterpret_cast<const float*>(cuts + kMaxClusters);
  const int32_t s = (int32_t)blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MassCut c = cuts[s];
  if (c.last <= s) return;
  const MassReq q = mass_req(a.plan, c.r, a.pool.page_size);
  const int32_t rel = c.kt * (2 * kMK) + (int32_t)threadIdx.x;
  if (rel >= q.n || !mass_seen(a, q, rel)) return;
  const int32_t page = mass_page(a.plan, q, rel, a.pool.page_size, a.pool.num_pages);
  if (page == a.pool.num_pages) return;  // reported by the producer
  float sum = recs[((int64_t)s * 2 + c.slot) * (2 * kMK) + threadIdx.x];
  // (a cluster between them without tiles has no record)
  for (int32_t k0 = s + 1; k0 <= c.last; k0 += 16) {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = k0 + k <= c.last && !(c.sparse && cuts[k0 + k].empty)
                 ? recs[((int64_t)(k0 + k) * 2) * (2 * kMK) + threadIdx.x]
                 : 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) sum += v[k];
  }
  mass_store(a, q, page, c.g, rel, sum);
}

template <int D>
cudaError_t launch_mass(const MassArgs& m, cudaStream_t stream) {
  const AttnArgs& a = m.attn;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap tq, tk;
  cuuint32_t es[4] = {1, 1, 1, 1};
  {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.num_qo_heads, (cuuint64_t)a.plan.num_tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.num_qo_heads * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)(kNQ / 2 / a.group)};
    if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)a.q, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int32_t ps = a.pool.page_size, br = std::min(ps, kMK);
  {
    const cuuint64_t rows = (cuuint64_t)a.pool.num_pages * 2 * a.pool.num_kv_heads * ps;
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)D / 64, rows / 8};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 2 * 8};
    cuuint32_t box[4] = {64, 8, 4, (cuuint32_t)br / 8};
    if (enc(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void*)a.pool.layer_base, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  static PerDeviceOnce setup;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = setup.get(dev, [dev](int* n) {
    const cudaError_t r = cudaFuncSetAttribute(mass_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               MassCfg<D>::SMEM);
    if (r != cudaSuccess) return r;
    return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  }, &sms);
  if (e != cudaSuccess) return e;
  const int32_t clusters = std::max(1, std::min(sms / 2, kMaxClusters));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
  cfg.blockDim = dim3(kThreadsMass, 1, 1);
  cfg.dynamicSmemBytes = MassCfg<D>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, mass_tc_kernel<D>, tq, tk, m, br);
  if (e != cudaSuccess) return e;
  count_launch();
  cfg.gridDim = dim3((unsigned)clusters, 1, 1);
  cfg.blockDim = dim3(2 * kMK, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, mass_join_kernel, m);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace

size_t mass_tc_ws_bytes() { return kMaxClusters * (sizeof(MassCut) + 2 * 2 * kMK * sizeof(float)); }

cudaError_t launch_mass_prefill_tc(const MassArgs& m, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_mass<256>(m, stream) : launch_mass<512>(m, stream);
}

}  // namespace pg
