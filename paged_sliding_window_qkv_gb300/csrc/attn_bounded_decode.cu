// Decode attention of bounded caches (sinks, window, optionally the weights of every key) on the
// tensor cores (tcgen05 + TMEM + TMA). Page sizes 8, 16, 32, ..., groups up to 16.
//
// A decode step reads every visible K and V row once and computes little with it, so the kernel
// is built to keep copies in flight and nothing else: the products are transposed so that keys and
// output columns are the 128 MMA rows and the group's query rows the 16 columns,
//   S^T = K Q^T   (M = 128 keys, N = 16, K = 16 d a step; A = K as it lands, K-major)
//   O^T = V^T P^T (M = 128 output columns, N = 16, K = 16 keys a step; A = V as it lands, MN-major)
// and a tile of 128 keys costs the tensor core about an eighth of the time its bytes take from
// HBM; the CUDA cores see 16 scores per key. O^T stays in TMEM for the segment.
//
// Work: a (request, KV head) segment's visible keys lie in boxes of 16 keys (8 at page size 8),
// sinks first, then the window (bounded.cuh); a tile is the next 128 rows of boxes, whatever
// positions they hold, so a few sinks cost one box and not a tile of their own (with tiles of
// consecutive keys 4 sinks beside a window of 1024 cost 10% of the call: a near-empty tile holds
// its ring slots as long as a full one). CTA s of S takes tiles [s U / S, (s + 1) U / S). A segment
// cut between CTAs leaves fp32 records (O / l, m, l) that the join kernel combines. (Smaller tiles
// for steps that leave SMs idle were slower: one request of 8001 keys at head_dim 512 took 24.6 us
// in tiles of 32 keys, whose unused rows have to be cleared, against 16.4.)
//
//   warps 0, 6  producers of K and of V: three 64 KB slots (128 keys x 256 d, one 4-D box per 16
//             keys and slot, all landing as [8 keys][64-d chunk][8 rows][128 B]) of one ring, in
//             the order K0 K1 V0 K2 V1 ...; warp 0 also the group's query rows per segment and a
//             header per tile (visible keys as bits, flags). (Six slots of 128 d, boxes of half the
//             bytes: 187 against 171 us on 64 requests of 8001 keys at head_dim 512.)
//   warp 1    MMA issuer: QK of tile i + 1 before PV of tile i, so a tile's softmax has a tile's
//             load time to finish
//   warps 2-5 softmax: a thread is a key (TMEM lane); 16 scores, exponentials against a per-row
//             reference with 2^64 headroom that moves only when a score outgrows it by 2^48 (so no
//             maximum is taken across keys in the common tile), P to shared memory; V rows of keys
//             that are not visible are zeroed (whatever they held); a segment's output leaves one
//             tile late, when its last PV is done anyway.
//
// Weights: the scores of visible keys go to the workspace (64 contiguous bytes a key at 16 heads),
// and the join kernel, which has the normalisers, adds each key's weights to its statistics in
// the same launch that combines the records.
//
// Every wait is bounded (a wait that runs out sets the device status word and the CTA leaves); the
// softmax warps agree on giving up before any barrier among themselves.
#include "bounded.cuh"
#include "mass.cuh"
#include "pg_internal.h"
#include "tc_ptx.cuh"

#include <math.h>

#include <algorithm>

namespace pg {
namespace {

constexpr int kT = 128;               // keys per tile
constexpr int kN = 16;                // MMA columns: query rows of the group, padded
constexpr int kThreadsDec = 224;
constexpr int kMaxCtas = 256;         // records are sized for at most this many CTAs
constexpr int kHdrs = 4;
constexpr float kRescale = 48.f, kHeadroom = 64.f;  // see attn_tc.cu
constexpr float kLn2f = 0.69314718055994531f, kLog2ef = 1.4426950408889634f;

constexpr int kFirst = 1, kLast = 2, kSplit = 4, kEnd = 8, kEmpty = 16, kRec1 = 32;

struct alignas(16) TileHdr {
  uint32_t vis[4];  // visible keys
  int32_t rel[16];  // key index (from the request's first key) of each box's first row
  int32_t flags, r, g, tok;
  int64_t slot0;    // slot of the request's first key, counted through the batch's page list
};

template <int D>
struct BdCfg {
  static constexpr int SD = 256;                   // d of a slot
  static constexpr int NC = SD / 64;               // 64-d chunks of a slot
  static constexpr int SLOT = kT * SD * 2;
  static constexpr int PARTS = D / SD;             // slots per tile of K, and of V
  static constexpr int NSLOT = 3;
  static constexpr int NQB = D == 256 ? 2 : 1;     // query buffers (segments)
  static constexpr int Q_BYTES = (D / 64) * kN * 128;  // [64-d chunk][16 rows][128 B]
  static constexpr int P_BYTES = 2 * kN * 128;         // [64-key chunk][16 rows][128 B]
  static constexpr int OFF_Q = NSLOT * SLOT;
  static constexpr int OFF_P = OFF_Q + NQB * Q_BYTES;
  static constexpr int OFF_HDR = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_RED = OFF_HDR + kHdrs * (int)sizeof(TileHdr);  // [4 warps][16]
  static constexpr int OFF_FIN = OFF_RED + 4 * kN * 4;                    // [16] (l, reference)
  static constexpr int OFF_BAR = OFF_FIN + kN * 8;
  // FULL, EMPTY; QFULL[2], QEMPTY[2], HFULL[4], HEMPTY[4], SFULL[2], SFREE[2], PFULL[2], PVDONE[2],
  // OFREE[2], DRAIN
  static constexpr int NBAR = 2 * NSLOT + 4 + 8 + 10 + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static constexpr uint32_t TM_O = 0, O_COLS = D / 128 * kN, TM_S = 2 * O_COLS;
  static constexpr uint32_t TM_COLS = TM_S + 2 * kN <= 128 ? 128 : 256;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct BdArgs {
  AttnArgs a;
  float* rec_o;     // [S][2][G][D]
  float* rec_ml;    // [S][2][G][2]
  int64_t* prefix;  // [R + 1] tiles before request r (all heads)
  int32_t box_rows;
  int32_t box_lg, page_lg;  // log2 of box_rows and of the page size (both powers of two)
};

// ------------------------------------------------------------------ PTX (one CTA)
// K and V are read once a step: their lines leave L2 first, so that scores and records stay for the join
// (64 requests of 8001 keys at head_dim 512: 176 -> 170 us, with weights 202 -> 197; 16: 63 -> 57).
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* tm, int c2, int c3, uint32_t bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(tm), "r"(0), "r"(c2), "r"(c3), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma1(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, p;\n .reg .u32 ln;\n mov.u32 ln, %%laneid;\n setp.eq.u32 e, ln, 0;\n setp.ne.b32 p, %3, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(acc), "n"(IDESC)
      : "memory");
}
__device__ __forceinline__ void commit1(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .u32 ln;\n mov.u32 ln, %%laneid;\n setp.eq.u32 e, ln, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : PG_R8(0), PG_R8(8)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      PG_W8(0), PG_W8(8)
      : "memory");
}
// barriers among the 128 softmax threads
__device__ __forceinline__ bool any4(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync4() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
// maximum over the warp
__device__ __forceinline__ float warp_max(float x) {
  const int32_t b = __float_as_int(x);
  const int32_t m = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7FFFFFFF));
  return __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
}

// The boxes of request r that its query sees, and the tiles they fill (one KV head).
struct ReqTiles {
  KeyWalk w;      // in boxes
  int32_t total;  // tiles
  int32_t tok, kvp0, kvp1, kv_len, ks0, sink;
  __device__ __forceinline__ bool sees(int32_t key) const {
    return key < w.hi && (key >= w.lo || key < sink);
  }
};
__device__ __forceinline__ ReqTiles req_tiles(const BdArgs& args, int32_t r) {
  const AttnArgs& a = args.a;
  const int4 e0 = __ldg(reinterpret_cast<const int4*>(a.plan.pair_tab) + 2 * r);
  const int4 e1 = __ldg(reinterpret_cast<const int4*>(a.plan.pair_tab) + 2 * r + 1);
  ReqTiles t;
  t.tok = e0.y;
  t.kvp0 = e1.x;
  t.kvp1 = e1.y;
  t.kv_len = e1.z;
  t.ks0 = e1.w;
  t.sink = a.window_left >= 0 ? a.num_sink : 0;
  t.w = key_walk(a.window_left, a.num_sink, t.ks0, t.kv_len, e0.w, e0.w, args.box_rows);
  const int32_t nbox = kT >> args.box_lg;
  t.total = (t.w.total + nbox - 1) / nbox;
  return t;
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreadsDec, 1)
bounded_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                      BdArgs args) {
  using C = BdCfg<D>;
  constexpr int NS = C::NSLOT, PARTS = C::PARTS;
  const AttnArgs& a = args.a;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gb = smem_raw + (base - raw);
  const uint32_t bars = base + C::OFF_BAR;
  auto FULL = [&](int s) { return bars + 8u * s; };
  auto EMPTY = [&](int s) { return bars + 8u * (NS + s); };
  const uint32_t QFULL = bars + 8u * (2 * NS), QEMPTY = QFULL + 16, HFULL = QFULL + 32, HEMPTY = HFULL + 32,
                 SFULL = HEMPTY + 32, SFREE = SFULL + 16, PFULL = SFULL + 32, PVDONE = SFULL + 48,
                 OFREE = SFULL + 64, DRAIN = SFULL + 80;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gb + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, a.status, a.wait_ns};
  TileHdr* const hdrs = reinterpret_cast<TileHdr*>(gb + C::OFF_HDR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t G = a.group, Hq = a.num_qo_heads, Hkv = a.pool.num_kv_heads, ps = a.pool.page_size;

  if (threadIdx.x == 32) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(QFULL + 8 * b, 1);
      mbar_init(QEMPTY + 8 * b, 1);
      mbar_init(SFULL + 8 * b, 1);
      mbar_init(SFREE + 8 * b, 4);
      mbar_init(PFULL + 8 * b, 4);
      mbar_init(PVDONE + 8 * b, 1);
      mbar_init(OFREE + 8 * b, 4);
    }
    for (int h = 0; h < kHdrs; ++h) {
      mbar_init(HFULL + 8 * h, 1);
      mbar_init(HEMPTY + 8 * h, 5);  // the softmax warps and the MMA issuer
    }
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // query and weight rows past the group stay zero
  if (warp >= 2 && warp < 6) {
    for (int i = threadIdx.x - 64; i < (C::NQB * C::Q_BYTES + 2 * C::P_BYTES) / 16; i += 128)
      *reinterpret_cast<uint4*>(gb + C::OFF_Q + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }
  // The producers find their tiles while the others set up, and (launched programmatically) while
  // the stream's previous kernel ends: a plan's metadata is written by copies alone, which no
  // programmatic launch overtakes. Everything else waits for that kernel.
  int32_t n = 0, r = 0;
  int64_t in_req = 0;
  constexpr int kHeld = 4;
  int64_t held[kHeld] = {0, 0, 0, 0};  // inclusive sums of the first requests' tiles
  if (warp == 0 || warp == 6) {
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_kv) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_q) : "memory");
    }
    const int32_t R = a.plan.num_req;
    const int64_t S = gridDim.x, s = blockIdx.x;
    // Tiles of every request (all heads) in scans of 32 requests: the total, and the request that
    // holds the CTA's first tile. The first scans' counts are loaded together and kept.
    auto tiles_of = [&](int32_t r) -> int64_t { return r < R ? (int64_t)req_tiles(args, r).total * Hkv : 0; };
    auto scan = [&](int64_t v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      return v;
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) held[j] = tiles_of(32 * j + lane);
    int64_t U = 0;
    for (int32_t c = 0; c < R; c += 32) {
      const int j = c / 32;
      const int64_t v = j == 0 ? held[0] : j == 1 ? held[1] : j == 2 ? held[2] : j == 3 ? held[3] : tiles_of(c + lane);
      const int64_t incl = U + scan(v);
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (k == j) held[k] = incl;
      U = __shfl_sync(0xffffffffu, incl, 31);
    }
    const int64_t u0 = s * U / S, u1 = (s + 1) * U / S;
    n = (int32_t)(u1 - u0);
    if (n > 0) {
      int64_t run = 0;  // tiles before request c
      for (int32_t c = 0; c < R; c += 32) {
        const int j = c / 32;
        const int64_t incl = j == 0   ? held[0]
                             : j == 1 ? held[1]
                             : j == 2 ? held[2]
                             : j == 3 ? held[3]
                                      : run + scan(tiles_of(c + lane));
        const uint32_t past = __ballot_sync(0xffffffffu, incl > u0);
        if (past) {
          const int f = __ffs(past) - 1;
          r = c + f;
          const int64_t before = __shfl_up_sync(0xffffffffu, incl, 1);
          in_req = u0 - __shfl_sync(0xffffffffu, lane == 0 ? run : before, f);
          break;
        }
        run = __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(C::TM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------ producers
    // Both walk the tiles; warp 0 issues K, the queries and the headers, warp 6 issues V. (One warp
    // for both took some 5 us a tile at head_dim 512 without any copy in it: the copies' issue.)
    const bool is_v = warp == 6;
    // the prefix for the join (CTA 0), once the stream's previous kernel, which may read the last one
    // in the same workspace, has ended
    auto write_prefix = [&]() {
      if (blockIdx.x != 0 || is_v) return;
      const int32_t R = a.plan.num_req;
      int64_t run = 0;
      for (int32_t c = 0; c < R; c += 32) {
        const int j = c / 32;
        int64_t incl;
        if (j < kHeld) {
          incl = j == 0 ? held[0] : j == 1 ? held[1] : j == 2 ? held[2] : held[3];
        } else {
          incl = c + lane < R ? (int64_t)req_tiles(args, c + lane).total * Hkv : 0;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          incl += run;
        }
        if (c + lane < R) args.prefix[c + lane + 1] = incl;
        run = __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) args.prefix[0] = 0;
    };
    bool ok = true;
    if (n == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      write_prefix();
      if (lane == 0 && !is_v) {
        hdrs[0].flags = kEmpty | kEnd;
        mbar_arrive(HFULL);
      }
    } else {
      const int br = args.box_rows, nbox = kT / br;
      const uint64_t policy = evict_first();
      // the tile that the iterator stands on
      ReqTiles q = req_tiles(args, r);
      int32_t g = (int32_t)(in_req / q.total), j = (int32_t)(in_req % q.total);
      int32_t nseg = 0;
      struct Tile {
        int32_t flags, r, g;
        int32_t rel, page, off;  // this lane's box: key index of its first row, page, row in the page
        bool live;               // the lane has a box
        ReqTiles q;
      };
      // describes tile i and steps on; the lane's page id is loaded here and used a tile later
      int32_t seg_split = 0;
      auto next = [&](int32_t i) {
        Tile t;
        if (i == 0 || j == 0) {
          const int32_t rest = q.total - j;
          seg_split = (j != 0 || rest > n - i) ? kSplit : 0;
          seg_split |= nseg > 0 ? kRec1 : 0;
          ++nseg;
          t.flags = kFirst;
        } else {
          t.flags = 0;
        }
        t.flags |= seg_split | (j == q.total - 1 || i == n - 1 ? kLast : 0) | (i == n - 1 ? kEnd : 0);
        t.r = r;
        t.g = g;
        t.q = q;
        const int32_t v = j * nbox + lane;
        t.live = lane < nbox && v < q.w.total;
        t.rel = t.live ? q.w.tile(v) << args.box_lg : 0;
        t.page = -1;
        t.off = t.rel & (ps - 1);
        if (t.live) {
          const int32_t pidx = q.kvp0 + (t.rel >> args.page_lg);
          t.page = (pidx < q.kvp1 && pidx < a.plan.num_page_ids) ? a.plan.page_ids[pidx] : -1;
        }
        if (++j == q.total && i + 1 < n) {
          j = 0;
          if (++g == Hkv) {
            g = 0;
            do q = req_tiles(args, ++r);
            while (q.total == 0);
          }
        }
        return t;
      };
      // PARTS slots of K or V, from the at-th of the CTA's stream of slots (K0 K1 V0 K2 V1 ...)
      auto load = [&](const Tile& t, bool good, int32_t at) {
        const uint32_t boxes = __ballot_sync(0xffffffffu, good);
        const int32_t row = (int32_t)((((int64_t)t.page * 2 + (is_v ? 1 : 0)) * Hkv + t.g) * ps + t.off);
        int slot = at % NS, round = at / NS;
        for (int p = 0; p < PARTS; ++p) {
          if (!__all_sync(0xffffffffu, mbar_wait_inline(EMPTY(slot), (round & 1) ^ 1, wc))) return false;
          if (lane == 0) mbar_expect_tx(FULL(slot), (uint32_t)__popc(boxes) * br * (C::SD * 2u));
          __syncwarp();
          if (good) tma_4d(base + slot * C::SLOT + lane * br * (C::SD * 2), &tm_kv, C::NC * p, row / 8, FULL(slot), policy);
          if (++slot == NS) { slot = 0; ++round; }
        }
        return true;
      };
      Tile cur = next(0);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      int32_t segs = 0;
      for (int32_t i = 0; ok && i < n; ++i) {
        const bool good = cur.live && cur.page >= 0 && cur.page < a.pool.num_pages;
        if (is_v) {
          const int32_t at = PARTS * (i == n - 1 ? 2 * i + 1 : 2 * i + 2);
          // the next tile's page ids load behind this tile's copies
          const Tile t = cur;
          if (i + 1 < n) cur = next(i + 1);
          ok = load(t, good, at);
          continue;
        }
        const bool first = cur.flags & kFirst;
        if (first) {
          const int qb = segs % C::NQB;
          ok = __all_sync(0xffffffffu, mbar_wait_inline(QEMPTY + 8 * qb, ((segs / C::NQB) & 1) ^ 1, wc));
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(QFULL + 8 * qb, (uint32_t)(G * D * 2));
          __syncwarp();
          if (lane < D / 64)
            tma_3d(base + C::OFF_Q + qb * C::Q_BYTES + lane * (kN * 128), &tm_q, lane * 64, cur.g * G, cur.q.tok,
                   QFULL + 8 * qb);
          ++segs;
        }
        ok = __all_sync(0xffffffffu, mbar_wait_inline(HEMPTY + 8 * (i % kHdrs), ((i / kHdrs) & 1) ^ 1, wc));
        if (!ok) break;
        const uint32_t boxes = __ballot_sync(0xffffffffu, good);
        if (__any_sync(0xffffffffu, cur.live && !good) && lane == 0) atomicOr(a.status, kStatusBounds);
        uint32_t vis[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int k = 32 * w + lane, box = k >> args.box_lg;
          const int32_t key = cur.q.ks0 + __shfl_sync(0xffffffffu, cur.rel, box) + (k & (br - 1));
          vis[w] = __ballot_sync(0xffffffffu, ((boxes >> box) & 1u) && cur.q.sees(key));
        }
        TileHdr& h = hdrs[i % kHdrs];
        if (lane < nbox) h.rel[lane] = cur.rel;
        if (lane == 0) {
#pragma unroll
          for (int w = 0; w < 4; ++w) h.vis[w] = vis[w];
          h.flags = cur.flags;
          h.r = cur.r;
          h.g = cur.g;
          h.tok = cur.q.tok;
          h.slot0 = (int64_t)cur.q.kvp0 * ps;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(HFULL + 8 * (i % kHdrs));
        const Tile t = cur;
        if (i + 1 < n) cur = next(i + 1);
        ok = load(t, good, i == 0 ? 0 : PARTS * (2 * i - 1));
        if (i == 0) write_prefix();  // (behind the first copies)
      }
    }
    if (!ok) {
      const uint64_t t0 = globaltimer();  // the copies already issued land before the CTA leaves
      while (globaltimer() - t0 < 100000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t IDESC_QK = idesc_bf16(kT, kN, false);
    constexpr uint32_t IDESC_PV = idesc_bf16(kT, kN, false) | (1u << 15);  // A (V) is MN-major
    auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
      const bool w = lane == 0 ? mbar_wait_inline(bar, parity, wc) : false;
      return __shfl_sync(0xffffffffu, w ? 1 : 0, 0) != 0;
    };
    int slot = 0, round = 0;
    auto step = [&]() {
      if (++slot == NS) { slot = 0; ++round; }
    };
    int32_t segs = 0, flags = 0, pflags = 0, pseg = 0;
    bool end = false;
    for (int32_t i = 0;; ++i) {
      bool ok = true;
      pflags = flags;
      pseg = segs - 1;  // the segment of tile i - 1
      if (!end) {
        ok = wait1(HFULL + 8 * (i % kHdrs), (i / kHdrs) & 1);
        if (!ok) break;
        flags = hdrs[i % kHdrs].flags;
        __syncwarp();
        if (lane == 0) mbar_arrive(HEMPTY + 8 * (i % kHdrs));
        if (flags & kEmpty) break;
        if (flags & kFirst) {
          ok = wait1(QFULL + 8 * (segs % C::NQB), (segs / C::NQB) & 1);
          ++segs;
        }
        const int sb = i & 1;
        ok = ok && wait1(SFREE + 8 * sb, ((i >> 1) & 1) ^ 1);
        const uint32_t qb = base + C::OFF_Q + ((segs - 1) % C::NQB) * C::Q_BYTES;
        for (int p = 0; ok && p < PARTS; ++p) {
          ok = wait1(FULL(slot), round & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = sdesc(base + slot * C::SLOT, 16, C::NC * 1024);
          const uint64_t qd = sdesc(qb + p * C::NC * (kN * 128), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < C::SD / 16; ++kk)
            mma1<IDESC_QK>(tmem + C::TM_S + sb * kN, kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                           qd + (uint64_t)(((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4),
                           (p > 0 || kk > 0) ? 1u : 0u);
          commit1(EMPTY(slot));
          step();
        }
        if (!ok) break;
        commit1(SFULL + 8 * sb);
        if (flags & kLast) commit1(QEMPTY + 8 * ((segs - 1) % C::NQB));
      }
      if (i > 0) {
        const int32_t jt = i - 1;
        const int pb = jt & 1, ob = pseg & 1;
        ok = wait1(PFULL + 8 * pb, (jt >> 1) & 1);
        if (ok && (pflags & kFirst)) ok = wait1(OFREE + 8 * ob, ((pseg >> 1) & 1) ^ 1);
        for (int p = 0; ok && p < PARTS; ++p) {
          ok = wait1(FULL(slot), round & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t pd = sdesc(base + C::OFF_P + pb * C::P_BYTES, 16, 1024);
#pragma unroll
          for (int mb = 0; mb < C::SD / 128; ++mb) {  // 128 output columns: two chunks
            const uint64_t vd = sdesc(base + slot * C::SLOT + mb * 2048, 1024, C::NC * 1024);
#pragma unroll
            for (int kk = 0; kk < kT / 16; ++kk)
              mma1<IDESC_PV>(tmem + C::TM_O + ob * C::O_COLS + (p * (C::SD / 128) + mb) * kN,
                             vd + (uint64_t)((kk * 2 * C::NC * 1024) >> 4),
                             pd + (uint64_t)(((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4),
                             ((pflags & kFirst) && kk == 0) ? 0u : 1u);
          }
          commit1(EMPTY(slot));
          step();
        }
        if (!ok) break;
        commit1(PVDONE + 8 * pb);
      }
      if (end) break;
      end = flags & kEnd;
    }
    commit1(DRAIN);
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // the thread's key of each tile, and output column of 128
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    float* const red = reinterpret_cast<float*>(gb + C::OFF_RED);
    float2* const fin = reinterpret_cast<float2*>(gb + C::OFF_FIN);
    float l[NQ], ref[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) { l[x] = 0.f; ref[x] = -INFINITY; }
    bool ok = true;
    int32_t segs = 0;
    // the segment whose output is still to leave
    bool pending = false;
    int32_t p_tile = 0, p_flags = 0, p_g = 0, p_tok = 0, p_seg = 0;
    auto epilogue = [&]() {
      if (!__all_sync(0xffffffffu, mbar_wait(PVDONE + 8 * (p_tile & 1), (p_tile >> 1) & 1, wc))) {
        ok = false;
        return;
      }
      tc_fence_after();
      const int64_t row0 = (int64_t)p_tok * Hq + (int64_t)p_g * G;
      const int64_t rec = ((int64_t)blockIdx.x * 2 + ((p_flags & kRec1) ? 1 : 0)) * G;
      float inv[NQ];
#pragma unroll
      for (int x = 0; x < NQ; ++x) inv[x] = fin[x].x == 0.f ? 0.f : 1.f / fin[x].x;
#pragma unroll 1
      for (int p = 0; p < D / 128; ++p) {
        uint32_t o[kN];
        tmem_ld16(tl + C::TM_O + (p_seg & 1) * C::O_COLS + p * kN, o);
        tmem_wait_ld();
        const int d = p * 128 + row;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          if (x >= G) break;
          const float v = inv[x] == 0.f ? 0.f : __uint_as_float(o[x]) * inv[x];
          if (p_flags & kSplit) args.rec_o[(rec + x) * D + d] = v;
          else a.out[(row0 + x) * D + d] = __float2bfloat16_rn(v);
        }
      }
      if (row < G) {
        const float2 f = fin[row];
        if (p_flags & kSplit) *reinterpret_cast<float2*>(args.rec_ml + (rec + row) * 2) = make_float2(f.y, f.x);
        else if (a.lse) a.lse[row0 + row] = f.x != 0.f ? (f.y + log2f(f.x)) * kLn2f : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(OFREE + 8 * (p_seg & 1));
    };
    for (int32_t i = 0;; ++i) {
      const int b = i & 1, hb = i % kHdrs;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(HFULL + 8 * hb, (i / kHdrs) & 1, wc));
      struct { int32_t flags, g, tok; int64_t slot; uint32_t mine, all; } h{};
      if (ok) {
        const TileHdr& x = hdrs[hb];
        h.flags = x.flags;
        h.g = x.g;
        h.tok = x.tok;
        h.slot = x.slot0 + x.rel[row >> args.box_lg] + (row & (args.box_rows - 1));
        h.mine = x.vis[quarter];
        h.all = x.vis[0] & x.vis[1] & x.vis[2] & x.vis[3];
      }
      if (any4(!ok)) break;  // all four warps leave together
      if (h.flags & kEmpty) break;
      ok = __all_sync(0xffffffffu, mbar_wait_inline(SFULL + 8 * b, (i >> 1) & 1, wc));
      if (h.flags & kFirst) {
        ++segs;
#pragma unroll
        for (int x = 0; x < NQ; ++x) { l[x] = 0.f; ref[x] = -INFINITY; }
      }
      const bool vis = (h.mine >> lane) & 1u;
      uint32_t sv[kN];
      tc_fence_after();
      tmem_ld16(tl + C::TM_S + b * kN, sv);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(SFREE + 8 * b);
        mbar_arrive(HEMPTY + 8 * hb);
      }
      float t[NQ];
      bool over = false;
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        t[x] = vis ? __uint_as_float(sv[x]) * a.sm_scale_log2 : -INFINITY;
        over |= t[x] > ref[x] + kRescale;
      }
      if (a.logits && vis) {
        if (h.slot < a.logit_slots) {
          float* dst = a.logits + h.slot * Hq + h.g * G;
          if (NQ % 4 == 0 && G == NQ) {
#pragma unroll
            for (int x = 0; x + 3 < NQ; x += 4)
              *reinterpret_cast<float4*>(dst + x) = make_float4(t[x], t[x + 1], t[x + 2], t[x + 3]);
          } else {
#pragma unroll
            for (int x = 0; x < NQ; ++x)
              if (x < G) dst[x] = t[x];
          }
        } else {
          atomicOr(a.status, kStatusBounds);
        }
      }
      if (any4(over)) {
        // the rows' maximum over the tile, then references with headroom where it outgrew them
        float mine = -INFINITY;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          const float m = warp_max(t[x]);
          if (lane == x) mine = m;
        }
        if (lane < NQ) red[quarter * kN + lane] = mine;
        sync4();
        float al[NQ];
        bool scaled = false;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          const float m = fmaxf(fmaxf(red[x], red[kN + x]), fmaxf(red[2 * kN + x], red[3 * kN + x]));
          al[x] = 1.f;
          if (m > ref[x] + kRescale) {
            const float r2 = m + kHeadroom;
            if (ref[x] != -INFINITY) {
              // the root of the factor, applied twice: the step may pass 2^-126 (attn_tc.cu)
              al[x] = ex2(0.5f * (ref[x] - r2));
              l[x] = (l[x] * al[x]) * al[x];
              scaled = true;
            }
            ref[x] = r2;
          }
        }
        // O holds the segment's earlier tiles at the old references (uniform over the threads)
        if (scaled && !(h.flags & kFirst)) {
          const int32_t jt = i - 1;
          if (__all_sync(0xffffffffu, mbar_wait(PVDONE + 8 * (jt & 1), (jt >> 1) & 1, wc))) {
            tc_fence_after();
#pragma unroll 1
            for (int p = 0; p < D / 128; ++p) {
              uint32_t o[kN];
              const uint32_t at = tl + C::TM_O + ((segs - 1) & 1) * C::O_COLS + p * kN;
              tmem_ld16(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < NQ; ++x) o[x] = __float_as_uint((__uint_as_float(o[x]) * al[x]) * al[x]);
              tmem_st16(at, o);
            }
            tmem_wait_st();
          } else {
            ok = false;
          }
        }
        sync4();  // red has been read
      }
      // the P buffer is free once PV(i - 2) has read it
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(PVDONE + 8 * b, ((i >> 1) & 1) ^ 1, wc));
      unsigned char* const pp = gb + C::OFF_P + b * C::P_BYTES + (row >> 6) * (kN * 128) + (row & 7) * 2;
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const float e = ex2(t[x] - (ref[x] == -INFINITY ? 0.f : ref[x]));
        l[x] += e;
        *reinterpret_cast<__nv_bfloat16*>(pp + x * 128 + ((((row >> 3) & 7) ^ (x & 7)) << 4)) =
            __float2bfloat16_rn(e);
      }
      if (h.all != 0xFFFFFFFFu) {
        // V rows of keys that are not visible: zero once the copies have landed. The tile's V slots
        // follow K(i + 1) in the ring (K(0), K(1), V(0), ...; the last tile's follow V(i - 1))
        const int32_t before = PARTS * ((h.flags & kEnd) ? 2 * i + 1 : 2 * i + 2);
        // A parity wait tells a slot's phases apart only once the use before has been consumed. At
        // head_dim 512 that is K(i + 1) or V(i - 1), for the last tile K(i) or V(i - 1): scores of
        // tile i + 1 are complete after both (the MMAs run in order), PV of tile i - 1 after the latter.
        if (2 * PARTS <= NS) {
          // (the use before was K(i), or PV of the tile two before: both waited for above)
        } else if (!(h.flags & kEnd))
          ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(SFULL + 8 * (b ^ 1), ((i + 1) >> 1) & 1, wc));
        else if (i > 0)
          ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(PVDONE + 8 * (b ^ 1), ((i - 1) >> 1) & 1, wc));
#pragma unroll 1
        for (int p = 0; p < PARTS; ++p) {
          const int32_t at = before + p, sl = at % NS;
          ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(FULL(sl), (at / NS) & 1, wc));
          if (ok && !vis) {
            unsigned char* v = gb + sl * C::SLOT + (row >> 3) * (C::NC * 1024) + (row & 7) * 128;
#pragma unroll
            for (int c = 0; c < 8 * C::NC; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * 1024 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      fence_proxy_async();  // the MMA reads P (and cleared V rows) through the async proxy
      tc_fence_before();    // and O after any rescaling above
      __syncwarp();
      if (lane == 0) mbar_arrive(PFULL + 8 * b);
      if (pending && ok) epilogue();
      pending = false;
      if (h.flags & kLast) {
        // the row sums over the 128 keys of every tile, and the references, for the epilogue
        float mine = 0.f;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          float s = l[x];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == x) mine = s;
        }
        if (lane < NQ) red[quarter * kN + lane] = mine;
        sync4();
#pragma unroll
        for (int x = 0; x < NQ; ++x)
          if (row == x) fin[x] = make_float2((red[x] + red[kN + x]) + (red[2 * kN + x] + red[3 * kN + x]), ref[x]);
        sync4();
        pending = true;
        p_tile = i;
        p_flags = h.flags;
        p_g = h.g;
        p_tok = h.tok;
        p_seg = segs - 1;
      }
      if (h.flags & kEnd) break;
    }
    if (pending && ok) epilogue();
  }

  // the join's launch overlaps the last CTAs' ends (released earlier, its blocks would sit on the SMs
  // while the copies stream: 236 against 222 us on 64 requests of 8001 keys with weights)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(DRAIN, 0)) {
        if (globaltimer() - t0 > a.wait_ns) {
          atomicOr(a.status, kStatusTimeout);
          break;
        }
      }
    }
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TM_COLS) : "memory");
  }
}

// ------------------------------------------------------------------ join
// Where the records of a segment are: CTAs sa .. sb, the record slot of sa. (64-bit divisions only
// where the products need them: S is at most 256.)
struct SegRecs {
  int32_t sa, sb, slot_a;
  bool sparse;  // fewer tiles than CTAs: some of the CTAs hold none
};
__device__ __forceinline__ SegRecs seg_recs(int64_t first, int64_t tiles, int64_t U, int32_t S) {
  SegRecs s;
  if (U < (1 << 23)) {
    const uint32_t u = (uint32_t)U, f = (uint32_t)first, t = (uint32_t)tiles;
    s.sa = (int32_t)(((f + 1) * S - 1) / u);
    s.sb = (int32_t)(((f + t) * S - 1) / u);
    s.slot_a = (uint32_t)s.sa * u / (uint32_t)S < f ? 1 : 0;
  } else {
    s.sa = (int32_t)(((first + 1) * S - 1) / U);
    s.sb = (int32_t)(((first + tiles) * S - 1) / U);
    s.slot_a = (int64_t)s.sa * U / S < first ? 1 : 0;
  }
  s.sparse = U < S;
  return s;
}
__device__ __forceinline__ bool holds_tiles(const SegRecs& s, int32_t c, int64_t U, int32_t S) {
  if (!s.sparse) return true;
  const uint32_t u = (uint32_t)U;
  return (uint32_t)c * u / (uint32_t)S < (uint32_t)(c + 1) * u / (uint32_t)S;
}

// Blocks [0, R Hkv G D RG / 512): 512 / RG columns of one segment's records into its output
// (segments inside one CTA were written directly; a segment without keys gets zeros), four columns
// a thread and eight records in flight.
// Blocks from there on (weights): 256 keys of one request, two a thread, all heads. The scores and
// page ids load while the normalisers are taken from the records (eight lanes per head), or from
// lse where the segment was written directly.
constexpr int kJoinThreads = 128;
constexpr int kPer = 2;                         // keys of a thread
constexpr int kJoinKeys = kPer * kJoinThreads;  // keys of a weight block
constexpr int kJoinRecs = 8;
// RG: threads that share the records of four columns (4 where segments are cut into many, so that
// 32 records are in flight, else 1)
__host__ __device__ __forceinline__ int32_t join_parts(int32_t group, int32_t D, int32_t RG) {
  return (group * D * RG + 511) / 512;
}
template <int D, int RG>
__global__ void __launch_bounds__(kJoinThreads, 7) bounded_join_kernel(BdArgs args, int32_t S, int32_t key_blocks) {
  const AttnArgs& a = args.a;
  // (a following kernel launched programmatically may set up; it waits for this one)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t Hkv = a.pool.num_kv_heads, G = a.group, Hq = a.num_qo_heads, R = a.plan.num_req;
  const int64_t U = args.prefix[R];
  const int tid = threadIdx.x;
  const int32_t parts = join_parts(G, D, RG), merges = R * Hkv * parts;
  if ((int32_t)blockIdx.x < merges) {
    const int32_t seg = (int32_t)blockIdx.x / parts, r = seg / Hkv, g = seg % Hkv;
    constexpr int kCols = kJoinThreads / RG;
    __shared__ float4 s_acc[kJoinThreads];
    __shared__ float2 s_md[kJoinThreads];
    const int rg = tid / kCols;
    const int32_t idx = ((int32_t)blockIdx.x % parts) * kCols + tid % kCols;  // four columns of a row
    const int32_t row = idx / (D / 4), c4 = idx % (D / 4);
    const int64_t pre = args.prefix[r];
    const ReqTiles q = req_tiles(args, r);
    const int64_t row0 = (int64_t)q.tok * Hq + (int64_t)g * G;
    if (RG == 1 && row >= G) return;
    const bool mine = row < G && rg == 0;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (row0 + row) * D + 4 * c4);
    if (q.total == 0) {
      if (mine) {
        dst[0] = dst[1] = 0u;
        if (a.lse && c4 == 0) a.lse[row0 + row] = -INFINITY;
      }
      return;
    }
    const SegRecs s = seg_recs(pre + (int64_t)g * q.total, q.total, U, S);
    if (s.sa == s.sb) return;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float m2, float w2, float4 x, bool mean) {
      if (w2 == 0.f) return;  // saw no key (a NaN sum stays)
      const float mn = fmaxf(M, m2), so = exp2f(M - mn), e = exp2f(m2 - mn);
      const float w = mean ? w2 * e : e;  // records hold means, partial states sums
      acc.x = acc.x * so + w * x.x; acc.y = acc.y * so + w * x.y;
      acc.z = acc.z * so + w * x.z; acc.w = acc.w * so + w * x.w;
      den = den * so + w2 * e;
      M = mn;
    };
    for (int32_t c0 = s.sa + rg; row < G && c0 <= s.sb; c0 += RG * kJoinRecs) {
      float2 ml[kJoinRecs];
      float4 v[kJoinRecs];
#pragma unroll
      for (int k = 0; k < kJoinRecs; ++k) {
        const int32_t c = c0 + RG * k;
        const bool in = c <= s.sb && holds_tiles(s, c, U, S);
        const int64_t rb = ((int64_t)c * 2 + (c == s.sa ? s.slot_a : 0)) * G + row;
        ml[k] = in ? *reinterpret_cast<const float2*>(args.rec_ml + rb * 2) : make_float2(-INFINITY, 0.f);
        v[k] = in ? *reinterpret_cast<const float4*>(args.rec_o + rb * D + 4 * c4) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kJoinRecs; ++k) add(ml[k].x, ml[k].y, v[k], true);
    }
    if constexpr (RG > 1) {
      s_acc[tid] = acc;
      s_md[tid] = make_float2(M, den);
      __syncthreads();
      if (!mine) return;
#pragma unroll
      for (int k = 1; k < RG; ++k) {
        const float2 md = s_md[tid + k * kCols];
        add(md.x, md.y, s_acc[tid + k * kCols], false);
      }
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    dst[0] = pack_bf16(acc.x * inv, acc.y * inv);
    dst[1] = pack_bf16(acc.z * inv, acc.w * inv);
    if (a.lse && c4 == 0) a.lse[row0 + row] = den != 0.f ? (M + log2f(den)) * kLn2f : -INFINITY;
    return;
  }
  // ---- weights
  extern __shared__ __align__(16) float s_lse[];  // the request's normalisers, log2 units
  const int32_t ps = a.pool.page_size;
  const int32_t r = ((int32_t)blockIdx.x - merges) / key_blocks, kb = ((int32_t)blockIdx.x - merges) % key_blocks;
  const MassReq q = mass_req(a.plan, r, ps);
  if ((int64_t)kb * kJoinKeys >= q.n) return;
  const ReqTiles t = req_tiles(args, r);
  if (t.total == 0) return;
  const int64_t pre = args.prefix[r];
  const float* src[kPer];
  int32_t page[kPer];
  float4 x[kPer][4];
  // 16 heads: a key's scores are four vectors, on their way while the normalisers form; other head counts
  // load them one at a time behind that (64 requests of 8001 keys at head_dim 512: 196 us with 16 heads, 187
  // with 8, 419 with 32 over two KV heads; the bytes take 155, 155 and 310)
  const bool vec = Hq == 16;
  auto load = [&](int64_t k0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t k = k0 + i * kJoinThreads + tid;
      const int32_t rel = (int32_t)min(k, (int64_t)q.n - 1);
      const int64_t slot = (int64_t)q.kvp0 * ps + rel;
      const bool seen = k < q.n && t.sees(q.ks0 + rel) && slot < a.logit_slots;
      // (a page out of range was reported by the decode kernel)
      page[i] = seen ? mass_page(a.plan, q, rel, ps, a.pool.num_pages) : a.pool.num_pages;
      src[i] = a.logits + (seen ? slot * Hq : 0);
      if (vec && seen) {
#pragma unroll
        for (int v = 0; v < 4; ++v) x[i][v] = reinterpret_cast<const float4*>(src[i])[v];
      }
    }
  };
  load((int64_t)kb * kJoinKeys);
  // eight lanes per head, a record each at a time
  const int sub = tid & 7;
  for (int h0 = 0; h0 < Hq; h0 += kJoinThreads / 8) {
    const int h = h0 + (tid >> 3);
    float M = -INFINITY, den = 0.f, direct = 0.f;
    SegRecs s{0, 0, 0, false};
    if (h < Hq) {
      s = seg_recs(pre + (int64_t)(h / G) * t.total, t.total, U, S);
      if (s.sa == s.sb) {
        direct = a.lse[(int64_t)q.q0 * Hq + h] * kLog2ef;
      } else {
        for (int32_t c = s.sa + sub; c <= s.sb; c += 8) {
          const int64_t rb = ((int64_t)c * 2 + (c == s.sa ? s.slot_a : 0)) * G + h % G;
          const float2 ml = holds_tiles(s, c, U, S) ? *reinterpret_cast<const float2*>(args.rec_ml + rb * 2)
                                                    : make_float2(-INFINITY, 0.f);
          if (ml.y != 0.f) {
            const float mn = fmaxf(M, ml.x);
            den = den * exp2f(M - mn) + ml.y * exp2f(ml.x - mn);
            M = mn;
          }
        }
      }
    }
    float mx = M;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float d = den != 0.f ? den * exp2f(M - mx) : 0.f;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (h < Hq && sub == 0) s_lse[h] = s.sa == s.sb ? direct : mx + log2f(d);
  }
  __syncthreads();
  // (a graph's plan may have grown since the capture: the blocks stride over the keys)
  for (int64_t k0 = (int64_t)kb * kJoinKeys; k0 < q.n; k0 += (int64_t)key_blocks * kJoinKeys) {
    if (k0 != (int64_t)kb * kJoinKeys) load(k0);
    if (vec) {
      // the group's sums of four heads at a time: a group is 1, 2 or a multiple of 4 of them
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (page[i] >= a.pool.num_pages) continue;
        const int32_t rel = (int32_t)(k0 + i * kJoinThreads + tid);
        float run = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float4 z = *reinterpret_cast<const float4*>(s_lse + 4 * v);
          const float e[4] = {ex2(x[i][v].x - z.x), ex2(x[i][v].y - z.y), ex2(x[i][v].z - z.z), ex2(x[i][v].w - z.w)};
          if (G >= 4) {
            run += (e[0] + e[1]) + (e[2] + e[3]);
            if ((4 * v + 4) % G == 0) {
              mass_store(a, q, page[i], 4 * v / G, rel, run);
              run = 0.f;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              run += e[k];
              if ((k + 1) % G == 0) {
                mass_store(a, q, page[i], (4 * v + k) / G, rel, run);
                run = 0.f;
              }
            }
          }
        }
      }
    } else {
      for (int32_t g = 0; g < Hkv; ++g) {
        float sum[kPer] = {};
        for (int32_t h = g * G; h < (g + 1) * G; ++h) {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (page[i] < a.pool.num_pages) sum[i] += ex2(src[i][h] - s_lse[h]);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (page[i] < a.pool.num_pages)
            mass_store(a, q, page[i], g, (int32_t)(k0 + i * kJoinThreads + tid), sum[i]);
      }
    }
  }
}

size_t al16(size_t n) { return (n + 15) & ~(size_t)15; }

// CTAs whose records the workspace holds (one that runs alone cuts no segment and leaves none).
int32_t record_room(const AttnArgs& a, int32_t D) {
  const size_t prefix = al16((size_t)(a.plan.num_req + 1) * 8), cta = (size_t)2 * a.group * (D + 2) * sizeof(float);
  const size_t room = a.ws_bytes > prefix ? (a.ws_bytes - prefix) / cta : 0;
  return (int32_t)std::min<size_t>(std::max<size_t>(room, 1), kMaxCtas);
}

template <int D, int NQ>
cudaError_t launch_bd(const AttnArgs& a, cudaStream_t stream) {
  using C = BdCfg<D>;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const int32_t ps = a.pool.page_size, Hkv = a.pool.num_kv_heads, G = a.group;
  CUtensorMap tq, tkv;
  cuuint32_t es[4] = {1, 1, 1, 1};
  {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.num_qo_heads, (cuuint64_t)a.plan.num_tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.num_qo_heads * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)G, 1};
    if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)a.q, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  const int32_t br = std::min(ps, 16);  // key rows per box
  {
    // (64 d, row within an 8-row group, 64-d chunk, 8-row group): a box is br rows of a slot
    const cuuint64_t rows = (cuuint64_t)a.pool.num_pages * 2 * Hkv * ps;
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)D / 64, rows / 8};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 2 * 8};
    cuuint32_t box[4] = {64, 8, (cuuint32_t)C::NC, (cuuint32_t)br / 8};
    if (enc(&tkv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void*)a.pool.layer_base, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  static PerDeviceOnce setup;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = setup.get(dev, [dev](int* n) {
    cudaError_t r = cudaFuncSetAttribute(bounded_decode_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM);
    if (r != cudaSuccess) return r;
    return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  }, &sms);
  if (e != cudaSuccess) return e;
  // as many CTAs as have tiles and room for their records
  const int32_t S = std::max(1, std::min(std::min(sms, record_room(a, D)), a.max_tiles));
  BdArgs b;
  b.a = a;
  b.box_rows = br;
  b.box_lg = 31 - __builtin_clz((unsigned)br);
  b.page_lg = 31 - __builtin_clz((unsigned)ps);
  unsigned char* ws = reinterpret_cast<unsigned char*>(a.ws_raw);
  b.prefix = reinterpret_cast<int64_t*>(ws);
  b.rec_ml = reinterpret_cast<float*>(ws + al16((size_t)(a.plan.num_req + 1) * 8));
  b.rec_o = b.rec_ml + (size_t)S * 2 * G * 2;
  // programmatic serialisation: the CTAs' set-up overlaps the end of the stream's previous kernel
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, 1, 1);
  cfg.blockDim = dim3(kThreadsDec, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, bounded_decode_kernel<D, NQ>, tq, tkv, b);
  if (e != cudaSuccess) return e;
  count_launch();
  const bool weigh = a.stats.mass != nullptr;
  const int32_t key_blocks = weigh ? (a.max_keys + kJoinKeys - 1) / kJoinKeys : 0;
  const int32_t segs = a.plan.num_req * Hkv;
  auto join = [&](auto kernel, int32_t RG) {
    const unsigned grid =
        (unsigned)((int64_t)segs * join_parts(G, D, RG) + (int64_t)a.plan.num_req * key_blocks);
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = weigh ? a.num_qo_heads * sizeof(float) : 0;
    return cudaLaunchKernelEx(&cfg, kernel, b, S, std::max(key_blocks, 1));
  };
  e = segs * 4 < S ? join(bounded_join_kernel<D, 4>, 4) : join(bounded_join_kernel<D, 1>, 1);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace

bool bounded_decode_supported(int32_t head_dim, int32_t group, int32_t page_size) {
  return (head_dim == 256 || head_dim == 512) && group >= 1 && group <= kN && page_size >= 8 &&
         (page_size & (page_size - 1)) == 0;
}

size_t bounded_decode_ws_bytes(int32_t num_req, int32_t group, int32_t head_dim, int32_t max_tiles) {
  const size_t S = (size_t)std::max(1, std::min(kMaxCtas, max_tiles));
  return al16((size_t)(num_req + 1) * 8) + S * 2 * group * 2 * 4 + S * 2 * group * head_dim * 4;
}

// pg_workspace_bytes of head_dim 512 may hold the records of fewer CTAs than have tiles. With room for
// less than half of them the chunked kernel is faster: 4 requests of 500 keys 35 against 65 us (17 with
// room for all), 64 of them 37 against 50 (33). With more it is not: one request of 8000 keys under a window
// of 1023, 10 tiles and room for 7 CTAs, 35 against 21 us.
bool bounded_decode_fits(const AttnArgs& a, int32_t head_dim) {
  if (a.logits) return true;  // (its workspace has them all)
  static PerDeviceOnce device;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return true;
  if (device.get(dev, [dev](int* v) { return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev); }, &sms) !=
      cudaSuccess)
    return true;
  int64_t tiles = a.max_tiles;
  if (a.window_left >= 0) {
    const int64_t seen = ((int64_t)a.window_left + a.num_sink + kT) / kT + 1;
    tiles = std::min(tiles, seen * a.plan.num_req * a.pool.num_kv_heads);
  }
  return 2 * (int64_t)record_room(a, head_dim) >= std::min<int64_t>(tiles, sms);
}

cudaError_t launch_bounded_decode(const AttnArgs& a, int32_t head_dim, cudaStream_t stream) {
  if (a.plan.num_req == 0) return cudaSuccess;
  // the fewest softmax rows that hold the group
  if (head_dim == 256) {
    if (a.group <= 2) return launch_bd<256, 2>(a, stream);
    if (a.group <= 4) return launch_bd<256, 4>(a, stream);
    if (a.group <= 8) return launch_bd<256, 8>(a, stream);
    return launch_bd<256, 16>(a, stream);
  }
  if (a.group <= 4) return launch_bd<512, 4>(a, stream);
  if (a.group <= 8) return launch_bd<512, 8>(a, stream);
  return launch_bd<512, 16>(a, stream);
}

}  // namespace pg
