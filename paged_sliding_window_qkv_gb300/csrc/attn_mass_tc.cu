// Accumulated attention weights of a prefill step on the tensor cores (tcgen05 + TMEM + TMA): the
// second pass behind the attention (attn_mass.cu says what is summed). Page sizes 8, 16, 32, ...
//
// S^T = K Q^T with keys as MMA rows: a key is a TMEM lane, so its sum over query rows runs along
// one thread's own columns, in registers, in one fixed order and without atomics.
//
// A unit is (request, KV head, 256 keys, a range of query tiles), one cluster of two CTAs, MMAs in
// the 2-SM form (M = 256 keys, N = 256 query rows, K = 16). CTA c keeps its 128 keys of K in
// shared memory for the whole unit (64 or 128 KB) and streams its half (128 rows) of every query
// tile through a ring of 16 KB stages (128 rows x 64 d). Two 256-column score buffers fill TMEM,
// so the sums of one tile overlap the products of the next. A query byte is used for 256 keys:
// the MMAs (D x 8 clocks per tile and SM) ask the ring for 32 bytes a clock from L2; with 128 keys
// they would ask for 64, which L2 does not give all SMs at once.
//
//   warp 0     producer: the unit's K once (one 4-D box per page and 256 d), then the query tiles
//   warp 1     MMA issuer (leader CTA)
//   warps 2-9  sums: two warps per TMEM lane quarter, 128 columns each; exp2(s c - lse) on fp32
//              pairs, masked on boundary tiles only. A tile's 128 terms are summed in four
//              accumulators and then added to the unit's sum with a compensated addition.
//
// Units of one query range follow one another in the grid (they read the same query tiles through
// L2), the last range first: it has the most keys. Each unit leaves its sums in the workspace; a
// small kernel adds a key's ranges in order and updates the statistics.
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

template <int D>
struct MassCfg {
  static constexpr int KP = D / 256;             // 256-d parts of a key row
  static constexpr int CH = D / 64;              // ring stages per query tile
  static constexpr int NS = D == 256 ? 8 : 5;    // ring stages
  static constexpr int K_BYTES = kMK * D * 2;
  static constexpr int OFF_Q = K_BYTES;
  static constexpr int OFF_LSE = OFF_Q + NS * kStage;      // [2 tile parities][256] -lse, log2 units
  static constexpr int OFF_X = OFF_LSE + 2 * kNQ * 4;      // [2 halves][128] final sums
  static constexpr int OFF_BAR = OFF_X + 2 * kMK * 4;
  // FULL[NS], EMPTY[NS], KFULL, AFULL[2], AEMPTY[2], LSE[2 halves][2 parities], PAIR[4], DRAIN
  static constexpr int NBAR = 2 * NS + 1 + 4 + 4 + 4 + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreadsMass, 1)
mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               MassArgs m, int32_t key_tiles, int32_t box_rows) {
  using C = MassCfg<D>;
  constexpr int NS = C::NS, CH = C::CH;
  const AttnArgs& a = m.attn;
  const PlanDev& pl = a.plan;
  const int32_t Hkv = a.pool.num_kv_heads, ps = a.pool.page_size, G = a.group, Hq = a.num_qo_heads;

  // ---- the unit: cluster id = ((range, request), KV head, key tile), the last range first
  int32_t id = (int32_t)blockIdx.x >> 1;
  const int32_t kt = id % key_tiles;
  id /= key_tiles;
  const int32_t g = id % Hkv;
  id /= Hkv;
  const int32_t r = id % pl.num_req;
  const int32_t c = m.splits - 1 - id / pl.num_req;
  const MassReq q = mass_req(pl, r, ps);
  const MassTiles mt = mass_tiles(a, q, kt);
  const int32_t t_lo = max(mt.first, c * m.chunk), t_hi = min(mt.end, (c + 1) * m.chunk);
  if (t_lo >= t_hi) return;  // both CTAs of the cluster
  const int32_t ntiles = t_hi - t_lo;

  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::OFF_BAR;
  auto FULL = [&](int s) { return bars + 8u * s; };
  auto EMPTY = [&](int s) { return bars + 8u * (NS + s); };
  const uint32_t KFULL = bars + 8u * (2 * NS), AFULL = KFULL + 8, AEMPTY = AFULL + 16,
                 LSEB = AEMPTY + 16, PAIR = LSEB + 32, DRAIN = PAIR + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, a.status, a.wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  auto LEAD = [&](uint32_t bar) { return mapa(bar, 0); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(FULL(s), 2);  // one arrival (with its byte count) from each CTA's producer
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(KFULL, 2);
    for (int b = 0; b < 2; ++b) {
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
  const int32_t TQ = kNQ / G;                              // tokens per query tile
  const int32_t rel0 = kt * (2 * kMK) + (int32_t)rank * kMK;  // this CTA's first key

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    {
      // K: lane l takes page boxes l, l + 32, ..., every 256-d part of each
      const int nbox = kMK / box_rows;
      uint32_t bytes = 0u;
      bool bad = false;
      for (int b = lane; b < nbox; b += 32) {
        const int32_t rel = rel0 + b * box_rows;
        if (rel >= q.n) continue;
        if (mass_page(pl, q, rel, ps, a.pool.num_pages) == a.pool.num_pages) bad = true;
        else bytes += (uint32_t)(C::KP * box_rows) * 512u;
      }
      for (int o = 16; o > 0; o >>= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, o);
      if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kStatusBounds);
      if (lane == 0) mbar_expect_tx_cl_relaxed(LEAD(KFULL), bytes);
      __syncwarp();
      for (int b = lane; b < nbox; b += 32) {
        const int32_t rel = rel0 + b * box_rows;
        if (rel >= q.n) continue;
        const int32_t page = mass_page(pl, q, rel, ps, a.pool.num_pages);
        if (page == a.pool.num_pages) continue;
        const int32_t row = (int32_t)(((int64_t)page * 2 * Hkv + g) * ps + rel % ps);
        for (int pp = 0; pp < C::KP; ++pp)
          tma_load_4d(base + pp * (kMK * 512) + b * box_rows * 512, &tm_k, 0, 0, pp * 4, row / 8,
                      LEAD(KFULL));
      }
      __syncwarp();
    }
    if (lane == 0) {
      int s = 0, round = 0;
      for (int32_t t = t_lo; ok && t < t_hi; ++t) {
        const int32_t tok = q.q0 + t * TQ + (int32_t)rank * (TQ / 2);
        for (int ch = 0; ch < CH; ++ch) {
          if (!mbar_wait_inline(EMPTY(s), (round & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          mbar_expect_tx_cl_relaxed(LEAD(FULL(s)), kStage);
          tma_load_3d(base + C::OFF_Q + s * kStage, &tm_q, ch * 64, g * G, tok, LEAD(FULL(s)));
          if (++s == NS) { s = 0; ++round; }
        }
      }
    }
    if (!__all_sync(0xffffffffu, ok)) {
      const uint64_t t0 = globaltimer();  // the copies already issued land before the CTA leaves
      while (globaltimer() - t0 < 100000ull) {
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the leader's)
    constexpr uint32_t IDESC = idesc_bf16(2 * kMK, kNQ, false);
    auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
      const bool w = lane == 0 ? mbar_wait_inline(bar, parity, wc) : false;
      return __shfl_sync(0xffffffffu, w ? 1 : 0, 0) != 0;
    };
    if (leader) {
      bool ok = wait1(KFULL, 0);
      int s = 0, round = 0;
      for (int32_t i = 0; ok && i < ntiles; ++i) {
        const int b = i & 1;
        ok = wait1(AEMPTY + 8 * b, ((i >> 1) & 1) ^ 1);
        for (int ch = 0; ok && ch < CH; ++ch) {
          ok = wait1(FULL(s), round & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = sdesc(base + (ch >> 2) * (kMK * 512) + (ch & 3) * 1024, 16, 4096);
          const uint64_t qd = sdesc(base + C::OFF_Q + s * kStage, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss<IDESC>(tmem + b * kNQ, kd + kk * 2, qd + kk * 2, (ch > 0 || kk > 0) ? 1u : 0u);
          mma_commit(EMPTY(s));
          if (++s == NS) { s = 0; ++round; }
        }
        if (ok) mma_commit(AFULL + 8 * b);
      }
      mma_commit(DRAIN);
    }
  } else {
    // ------------------------------------------------------------ sums
    const int quarter = warp & 3, h = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;                   // TMEM lane: this thread's key
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + h * (kNQ / 2);
    const int32_t rel = rel0 + row, j = q.ks0 + rel;
    const bool kvalid = rel < q.n;
    const int32_t W = a.window_left, sink = a.num_sink;
    const int gsh = __ffs(G) - 1;
    float* const lbuf = reinterpret_cast<float*>(gbase + C::OFF_LSE) + h * (kNQ / 2);
    // -lse (log2 units) of this thread's column of tile t; -inf: not a row of the request
    const int col = h * (kNQ / 2) + row;
    auto fetch = [&](int32_t t) -> float {
      const int32_t tk = t * TQ + (col >> gsh);
      if (t >= t_hi || tk >= q.len) return -INFINITY;
      return a.lse[(int64_t)(q.q0 + tk) * Hq + g * G + (col & (G - 1))] * -1.4426950408889634f;
    };
    float nxt = fetch(t_lo);
    float sum = 0.f, comp = 0.f;
    bool ok = true;
    const float2 sc = make_float2(a.sm_scale_log2, a.sm_scale_log2);
    for (int32_t i = 0; ok && i < ntiles; ++i) {
      const int b = i & 1;
      const int32_t t = t_lo + i;
      // this half's 128 values; the barrier of this parity also shows that all four warps are past
      // tile i - 1, so tile i + 1's values may replace it
      lbuf[b * kNQ + row] = nxt;
      nxt = fetch(t + 1);
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
      const int32_t p0 = q.sp + tk0, p1 = p0 + ntk - 1;
      const bool interior =
          __all_sync(0xffffffffu, tk0 + ntk <= q.len && kvalid && j <= p0 && (W < 0 || p1 - j <= W || j < sink));
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
            const float2 e0 = __ffma2_rn(make_float2(__uint_as_float(sv[4 * k]), __uint_as_float(sv[4 * k + 1])),
                                         sc, make_float2(l4.x, l4.y));
            const float2 e1 = __ffma2_rn(make_float2(__uint_as_float(sv[4 * k + 2]), __uint_as_float(sv[4 * k + 3])),
                                         sc, make_float2(l4.z, l4.w));
            s2[0] = __fadd2_rn(s2[0], make_float2(ex2(e0.x), ex2(e0.y)));
            s2[1] = __fadd2_rn(s2[1], make_float2(ex2(e1.x), ex2(e1.y)));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k) {
            const int32_t tk = tk0 + ((cb + k) >> gsh), p = q.sp + tk;
            const bool vis = tk < q.len && kvalid && j <= p && (W < 0 || p - j <= W || j < sink);
            const float e = fmaf(__uint_as_float(sv[k]), a.sm_scale_log2, lbuf[b * kNQ + cb + k]);
            s2[k & 1].x += vis ? ex2(e) : 0.f;
          }
        }
      }
      const float part = (s2[0].x + s2[1].x) + (s2[0].y + s2[1].y);
      // compensated: the unit's sum may add many tiles (an infinite or NaN sum stays as it is)
      const float y = part - comp, z = sum + y;
      comp = isfinite(z) ? (z - sum) - y : 0.f;
      sum = z;
    }
    // the two column halves of a key
    float* xs = reinterpret_cast<float*>(gbase + C::OFF_X);
    if (ok) {
      xs[h * kMK + row] = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(PAIR + 8 * quarter);
      ok = __all_sync(0xffffffffu, mbar_wait(PAIR + 8 * quarter, 0, wc));
      const int64_t slot = (int64_t)q.kvp0 * ps + rel;
      if (ok && h == 0 && kvalid) {
        if (slot < m.partial_slots)
          m.partial[((int64_t)c * Hkv + g) * m.partial_slots + slot] = xs[row] + xs[kMK + row];
        else
          atomicOr(a.status, kStatusBounds);
      }
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

// One thread per key: the sums of the query ranges that see the key's tile, in order.
__global__ void __launch_bounds__(256) mass_join_kernel(MassArgs m, int32_t blocks_per_req) {
  const AttnArgs& a = m.attn;
  const int32_t r = (int32_t)blockIdx.x / blocks_per_req;
  const int32_t Hkv = a.pool.num_kv_heads, ps = a.pool.page_size;
  const MassReq q = mass_req(a.plan, r, ps);
  const int32_t rel = ((int32_t)blockIdx.x % blocks_per_req) * 256 + (int32_t)threadIdx.x;
  if (rel >= q.n) return;
  const MassTiles t = mass_tiles(a, q, rel / (2 * kMK));
  const int64_t slot = (int64_t)q.kvp0 * ps + rel;
  if (t.first >= t.end || slot >= m.partial_slots) return;
  const int32_t page = mass_page(a.plan, q, rel, ps, a.pool.num_pages);
  if (page == a.pool.num_pages) return;  // reported by the producer
  for (int32_t g = 0; g < Hkv; ++g) {
    float sum = 0.f;
    for (int32_t c = t.first / m.chunk; c <= (t.end - 1) / m.chunk && c < m.splits; ++c)
      sum += m.partial[((int64_t)c * Hkv + g) * m.partial_slots + slot];
    mass_store(a, q, page, g, rel, sum);
  }
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
  int dev = 0, unused = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = setup.get(dev, [](int*) {
    return cudaFuncSetAttribute(mass_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                MassCfg<D>::SMEM);
  }, &unused);
  if (e != cudaSuccess) return e;
  const int32_t key_tiles = (a.max_keys + 2 * kMK - 1) / (2 * kMK);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (int64_t)key_tiles * a.pool.num_kv_heads * a.plan.num_req * m.splits), 1, 1);
  cfg.blockDim = dim3(kThreadsMass, 1, 1);
  cfg.dynamicSmemBytes = MassCfg<D>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, mass_tc_kernel<D>, tq, tk, m, key_tiles, br);
  if (e != cudaSuccess) return e;
  count_launch();
  const int32_t blocks = (a.max_keys + 255) / 256;
  mass_join_kernel<<<(unsigned)(blocks * (int64_t)a.plan.num_req), 256, 0, stream>>>(m, blocks);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

MassSplit mass_split(int32_t num_req, int32_t num_kv_heads, int32_t group, int64_t num_tokens,
                     int32_t max_qo_len, int32_t max_keys) {
  // About four units per cluster even out their lengths; a range is at least two query tiles, so
  // that a unit's K load (as long as a tile's products) is not most of it, and at most 64.
  const int64_t tiles = num_tokens * group / kNQ + num_req;  // query tiles of one KV head
  const int64_t key_tiles = ((int64_t)max_keys + 2 * kMK - 1) / (2 * kMK);
  const int64_t work = tiles * key_tiles * num_kv_heads;
  MassSplit s;
  s.chunk = (int32_t)std::min<int64_t>(64, std::max<int64_t>(2, work / (76 * 4)));
  const int64_t longest = ((int64_t)max_qo_len * group + kNQ - 1) / kNQ;
  s.splits = (int32_t)((longest + s.chunk - 1) / s.chunk);
  s.units = key_tiles * num_kv_heads * num_req * s.splits;
  return s;
}

cudaError_t launch_mass_prefill_tc(const MassArgs& m, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 256 ? launch_mass<256>(m, stream) : launch_mass<512>(m, stream);
}

}  // namespace pg
