// What the two bounded-cache decode kernels share (attn_bounded_decode.cu over bf16 pools,
// attn_q8_decode.cu over 8-bit ones): the walk over a step's tiles, the records that the join combines,
// and the PTX of a CTA on its own.
#pragma once

#include "bounded.cuh"
#include "pg_internal.h"
#include "tc_ptx.cuh"

namespace pg {

struct BdArgs {
  AttnArgs a;
  float* rec_o;     // [S][2][G][D]
  float* rec_ml;    // [S][2][G][2]
  int64_t* prefix;  // [R + 1] tiles before request r (all heads)
  int32_t box_rows;
  int32_t box_lg, page_lg;  // log2 of box_rows and of the page size (both powers of two)
};

// The join of a decode kernel's records (attn_bounded_decode.cu); S: the CTAs that the kernel ran on.
cudaError_t launch_bounded_join(const BdArgs& b, int32_t S, int32_t head_dim, cudaStream_t stream);
// CTAs whose records the workspace holds, and where the records lie in it.
int32_t bounded_record_room(const AttnArgs& a, int32_t head_dim, int32_t most);
size_t bounded_records_bytes(int32_t num_req, int32_t group, int32_t head_dim, int32_t ctas);
void bounded_records(const AttnArgs& a, int32_t S, BdArgs* b);

namespace {

constexpr int kT = 128;               // keys per tile
constexpr int kMaxCtas = 256;         // records are sized for at most this many CTAs
constexpr int kHdrs = 4;
constexpr float kRescale = 48.f, kHeadroom = 64.f;  // see attn_tc.cu
constexpr float kLn2f = 0.69314718055994531f, kLog2ef = 1.4426950408889634f;

constexpr int kFirst = 1, kLast = 2, kSplit = 4, kEnd = 8, kEmpty = 16, kRec1 = 32;

// ------------------------------------------------------------------ PTX (one CTA)
// K and V are read once a step: their lines leave L2 first, so that scores and records stay for the join
// (64 requests of 8001 keys at head_dim 512: 176 -> 170 us, with weights 202 -> 197; 16: 63 -> 57; 64 of up to
// 16384 keys in 8 bits 112 -> 104).
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
__device__ __forceinline__ void commit1(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .u32 ln;\n mov.u32 ln, %%laneid;\n setp.eq.u32 e, ln, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : PG_R8(0) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), PG_W8(0)
               : "memory");
}
// barriers among the 128 threads of a softmax set
__device__ __forceinline__ bool any_of(int bar, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(bar)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_set(int bar) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(bar) : "memory"); }
// The warp's maxima (SUM: sums) of CQ values a lane: lane i returns that of value set_col<CQ>(i). Halves
// the values at each exchange, so CQ of them cost about CQ + log2(32 / CQ) shuffles.
template <int CQ>
__device__ __forceinline__ int set_col(int lane) { return lane / (32 / CQ); }
template <int CQ, bool SUM>
__device__ __forceinline__ float warp_reduce(const float* x, int lane) {
  float v[CQ];
#pragma unroll
  for (int k = 0; k < CQ; ++k) v[k] = x[k];
  auto two = [](float p, float q) { return SUM ? p + q : fmaxf(p, q); };
  int mask = 16;
#pragma unroll
  for (int w = CQ; w > 1; w /= 2, mask /= 2) {
    const bool upper = lane & mask;
#pragma unroll
    for (int k = 0; k < w / 2; ++k) {
      const float got = __shfl_xor_sync(0xffffffffu, upper ? v[k] : v[k + w / 2], mask);
      v[k] = two(upper ? v[k + w / 2] : v[k], got);
    }
  }
#pragma unroll
  for (int m = 16 / CQ; m > 0; m /= 2) v[0] = two(v[0], __shfl_xor_sync(0xffffffffu, v[0], m));
  return v[0];
}

// What the kernel reads may come from the stream's previous kernel, unless it runs beside that one: then
// it only ends behind it, so that the stream's order holds for what follows.
__device__ __forceinline__ void wait_previous(const AttnArgs& a) {
  if (a.beside == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void wait_beside(const AttnArgs& a) {
  if (a.beside != 0) asm volatile("griddepcontrol.wait;" ::: "memory");
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

constexpr int kHeld = 4;  // scans of 32 requests whose tile counts stay in registers

// The tiles of CTA blockIdx.x: how many, and where the first is (request r, its in_req-th tile over all
// heads). held receives the inclusive sums of the first requests' tiles. Called by a whole warp.
__device__ __forceinline__ int32_t find_tiles(const BdArgs& args, int lane, int64_t* held, int32_t* r,
                                              int64_t* in_req) {
  const int32_t R = args.a.plan.num_req, Hkv = args.a.pool.num_kv_heads;
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
  const int32_t n = (int32_t)(u1 - u0);
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
        *r = c + f;
        const int64_t before = __shfl_up_sync(0xffffffffu, incl, 1);
        *in_req = u0 - __shfl_sync(0xffffffffu, lane == 0 ? run : before, f);
        break;
      }
      run = __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  return n;
}
// The inclusive sums of all requests' tiles, for the join (one warp of one CTA).
__device__ __forceinline__ void write_tile_prefix(const BdArgs& args, int lane, const int64_t* held) {
  const int32_t R = args.a.plan.num_req;
  int64_t run = 0;
  for (int32_t c = 0; c < R; c += 32) {
    const int j = c / 32;
    int64_t incl;
    if (j < kHeld) {
      incl = j == 0 ? held[0] : j == 1 ? held[1] : j == 2 ? held[2] : held[3];
    } else {
      incl = c + lane < R ? (int64_t)req_tiles(args, c + lane).total * args.a.pool.num_kv_heads : 0;
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
}

// The tiles of a CTA in order: one per next(), each lane with one box of it.
struct Tile {
  int32_t flags, r, g;
  int32_t rel, page, off;  // this lane's box: key index of its first row, page, row in the page
  bool live;               // the lane has a box
  ReqTiles q;
};
struct TileWalk {
  const BdArgs& args;
  const int lane;
  const int32_t n;
  int32_t r, g, j, nseg = 0, seg_split = 0;
  ReqTiles q;  // of the request that the walk stands on
  __device__ __forceinline__ TileWalk(const BdArgs& args_, int lane_, int32_t n_, int32_t r_, int64_t in_req)
      : args(args_), lane(lane_), n(n_), r(r_), q(req_tiles(args_, r_)) {
    g = (int32_t)(in_req / q.total);
    j = (int32_t)(in_req % q.total);
  }
  // describes tile i and steps on; the lane's page id is loaded here and used a tile later
  __device__ __forceinline__ Tile next(int32_t i) {
    const AttnArgs& a = args.a;
    const int nbox = kT >> args.box_lg;
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
    t.off = t.rel & (a.pool.page_size - 1);
    if (t.live) {
      const int32_t pidx = q.kvp0 + (t.rel >> args.page_lg);
      t.page = (pidx < q.kvp1 && pidx < a.plan.num_page_ids) ? a.plan.page_at(pidx) : -1;
    }
    if (++j == q.total && i + 1 < n) {
      j = 0;
      if (++g == a.pool.num_kv_heads) {
        g = 0;
        do q = req_tiles(args, ++r);
        while (q.total == 0);
      }
    }
    return t;
  }
};

}  // namespace
}  // namespace pg
