// Decode attention over 8-bit caches on the tensor cores (tcgen05 kind::f8f6f4 + TMEM + TMA).
// Power-of-two page sizes from 16 on, groups up to 16.
//
// A decode step reads every visible row once, and half the bytes of a bf16 cache leave half the time:
// converting 8-bit rows to 16 bits on the way to the tensor cores would cost the CUDA cores a
// conversion per element, more than that time. So the codes are multiplied as they land, and it is
// the few numbers that meet them that are split into 8-bit terms:
//   q = 2^e (a0 + a1 / 16)                  a0 = e4m3(q 2^-e), a1 = e4m3(16 (q 2^-e - a0))
//   S^T = K [a0 a1]^T  (M = 128 keys, N = the group's rows twice, K = 32 d a step)
//   s = 2^(e + k) (S0 + S1 / 16)            k: the exponent of the key's K row
//   P = 2^(s + v - R) = p0 + p1 / 16 + p2 / 256   v: of its V row; s in log2 units
//   O^T = V^T [p0 p1 p2]^T  (M = 128 output columns, N = the rows three times, K = 32 keys a step)
// Two terms hold a bf16 query exactly (8 bits of significand) down to 2^-15 of the row's largest
// element; three hold a weight to 12 bits. The terms only widen N, which at these sizes costs nothing:
// an instruction's time is that of reading A (the codes) from shared memory.
//
// e4m3 reaches from 2^-9 to 448, so R must stand near the row's largest s + v, not 2^48 off as in the
// bf16 kernels: it moves when an exponent outgrows it, to leave 4.8 octaves of room, and weights are
// cut off 2^-22 below the largest. The row sum keeps its own reference (of s alone) and adds the
// unrounded weights.
//
// Work, walk, records and join are those of attn_bounded_decode.cu; a ring slot is a tile of K or V
// (128 keys x head_dim codes: three slots of 64 KB, or six of 32 KB), in the order K0 K1 V0 K2 V1 ...
//   warps 0, 6  producers of K (with a header a tile) and of V: one 4-D box per 16 keys
//   warp 7      the group's query rows into their terms, a segment ahead as far as its buffer allows
//   warp 1      MMA issuer: QK of tile i + 1 before PV of tile i
//   warps 2-5   softmax: a thread is a key; its row scales load a tile ahead
// Every wait is bounded, as there.
#include "bounded_decode.cuh"
#include "q8.cuh"

#include <math.h>

#include <algorithm>

namespace pg {
namespace {

constexpr int kThreadsQ8 = 256;
constexpr int kQs = 4;  // segments whose query scales are kept
constexpr int kBox = 16, kBoxes = kT / kBox;  // key rows of a box, boxes of a tile
// P is at most 448 where a weight stands kRoom octaves above its reference; a reference is set kLead
// above the largest weight (P = 2^(8 - kLead) there).
constexpr float kTop = 8.f, kLead = 4.f, kRoom = 0.8f;

struct alignas(16) Q8Hdr {
  uint32_t vis[4];       // visible keys
  int32_t row[kBoxes];   // each box's first K row of the layer (-1: not loaded)
  int32_t flags, g, tok;
};

// NR: rows of a term (8 or 16, the group padded)
template <int D, int NR>
struct Q8Cfg {
  static constexpr int NC = D / 128;            // 128-d chunks of a row
  static constexpr int SLOT = kT * D;
  static constexpr int NSLOT = D == 256 ? 6 : 3;
  static constexpr int QN = 2 * NR;             // columns of S: two terms
  static constexpr int PN = NR == 8 ? 32 : 48;  // of O: three terms (N is a multiple of 16)
  static constexpr int NQB = D == 256 ? 2 : 1;  // query buffers (segments)
  static constexpr int Q_BYTES = NC * QN * 128; // [128-d chunk][QN rows][128 B]
  static constexpr int P_BYTES = PN * 128;      // [PN rows][128 keys]
  static constexpr int OFF_Q = NSLOT * SLOT;
  static constexpr int OFF_P = OFF_Q + NQB * Q_BYTES;
  static constexpr int OFF_QS = OFF_P + 2 * P_BYTES;                 // [kQs][16] query scales
  static constexpr int OFF_HDR = OFF_QS + kQs * 16 * 4;
  static constexpr int OFF_RED = OFF_HDR + kHdrs * (int)sizeof(Q8Hdr);  // [2][4 warps][16]
  static constexpr int OFF_FIN = OFF_RED + 2 * 4 * 16 * 4;           // [16] (l, its reference, P's)
  static constexpr int OFF_BAR = OFF_FIN + 16 * 16;
  // FULL, EMPTY; QFULL[2], QEMPTY[2], HFULL[4], HEMPTY[4], SFULL[2], SFREE[2], PFULL[2], PVDONE[2],
  // OFREE[2], DRAIN, QS[4]
  static constexpr int NBAR = 2 * NSLOT + 4 + 8 + 10 + 1 + kQs;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static constexpr uint32_t TM_O = 0, O_COLS = NC * PN, TM_S = 2 * O_COLS;
  static constexpr uint32_t TM_COLS = TM_S + 2 * QN <= 256 ? 256 : 512;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(TM_S + 2 * QN <= 512, "tensor memory");
};

struct Q8Args {
  BdArgs b;
  const uint8_t* scales;  // of the layer
};

// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 accumulate.
constexpr uint32_t idesc_e4m3(int N, bool a_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kT >> 4) << 24);
}
template <uint32_t IDESC>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, p;\n .reg .u32 ln;\n mov.u32 ln, %%laneid;\n setp.eq.u32 e, ln, 0;\n setp.ne.b32 p, %3, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(acc), "n"(IDESC)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (N >= 32) {
    tmem_ld32(taddr, r);
    if constexpr (N > 32) tmem_ld<N - 32>(taddr + 32, r + 32);
  } else {
    tmem_ld16(taddr, r);
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  if constexpr (N >= 32) {
    tmem_st32(taddr, r);
    if constexpr (N > 32) tmem_st<N - 32>(taddr + 32, r + 32);
  } else {
    tmem_st16(taddr, r);
  }
}
// two e4m3 numbers, the first in the low byte, and what they stand for
__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

template <int D, int NQ, int NR>
__global__ void __launch_bounds__(kThreadsQ8, 1)
q8_decode_kernel(const __grid_constant__ CUtensorMap tm_kv, Q8Args qa) {
  using C = Q8Cfg<D, NR>;
  constexpr int NS = C::NSLOT, NC = C::NC;
  const BdArgs& args = qa.b;
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
                 OFREE = SFULL + 64, DRAIN = SFULL + 80, QSCALE = SFULL + 88;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gb + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const WaitCtx wc{abort_flag, a.status, a.wait_ns};
  Q8Hdr* const hdrs = reinterpret_cast<Q8Hdr*>(gb + C::OFF_HDR);
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
      mbar_init(HEMPTY + 8 * h, 6);  // the softmax warps, the query warp and the MMA issuer
    }
    for (int q = 0; q < kQs; ++q) mbar_init(QSCALE + 8 * q, 1);
    mbar_init(DRAIN, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // query and weight rows past the group, and their scales, stay zero
  if (warp >= 2 && warp < 6) {
    for (int i = threadIdx.x - 64; i < (C::OFF_HDR - C::OFF_Q) / 16; i += 128)
      *reinterpret_cast<uint4*>(gb + C::OFF_Q + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
  }
  // The producers find their tiles while the others set up, and while the stream's previous kernel ends.
  int32_t n = 0, r = 0;
  int64_t in_req = 0;
  int64_t held[kHeld] = {0, 0, 0, 0};
  if (warp == 0 || warp == 6) {
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_kv) : "memory");
    n = find_tiles(args, lane, held, &r, &in_req);
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
    const bool is_v = warp == 6;
    bool ok = true;
    if (n == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (blockIdx.x == 0 && !is_v) write_tile_prefix(args, lane, held);
      if (lane == 0 && !is_v) {
        hdrs[0].flags = kEmpty | kEnd;
        mbar_arrive(HFULL);
      }
    } else {
      const uint64_t policy = evict_first();
      TileWalk walk(args, lane, n, r, in_req);
      // the tile's slot of K or V, the at-th of the CTA's stream of slots
      auto load = [&](const Tile& t, bool good, int32_t row, int32_t at) {
        const uint32_t boxes = __ballot_sync(0xffffffffu, good);
        const int slot = at % NS, round = at / NS;
        if (!__all_sync(0xffffffffu, mbar_wait_inline(EMPTY(slot), (round & 1) ^ 1, wc))) return false;
        if (lane == 0) mbar_expect_tx(FULL(slot), (uint32_t)__popc(boxes) * (kBox * D));
        __syncwarp();
        if (good) tma_4d(base + slot * C::SLOT + lane * (kBox * D), &tm_kv, 0, row / 8, FULL(slot), policy);
        return true;
      };
      Tile cur = walk.next(0);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int32_t i = 0; ok && i < n; ++i) {
        const bool good = cur.live && cur.page >= 0 && cur.page < a.pool.num_pages;
        const int32_t row = (int32_t)((((int64_t)cur.page * 2 + (is_v ? 1 : 0)) * Hkv + cur.g) * ps + cur.off);
        if (is_v) {
          const Tile t = cur;
          if (i + 1 < n) cur = walk.next(i + 1);
          ok = load(t, good, row, i == n - 1 ? 2 * i + 1 : 2 * i + 2);
          continue;
        }
        ok = __all_sync(0xffffffffu, mbar_wait_inline(HEMPTY + 8 * (i % kHdrs), ((i / kHdrs) & 1) ^ 1, wc));
        if (!ok) break;
        const uint32_t boxes = __ballot_sync(0xffffffffu, good);
        if (__any_sync(0xffffffffu, cur.live && !good) && lane == 0) atomicOr(a.status, kStatusBounds);
        uint32_t vis[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int k = 32 * w + lane, box = k / kBox;
          const int32_t key = cur.q.ks0 + __shfl_sync(0xffffffffu, cur.rel, box) + (k & (kBox - 1));
          vis[w] = __ballot_sync(0xffffffffu, ((boxes >> box) & 1u) && cur.q.sees(key));
        }
        Q8Hdr& h = hdrs[i % kHdrs];
        if (lane < kBoxes) h.row[lane] = good ? row : -1;
        if (lane == 0) {
#pragma unroll
          for (int w = 0; w < 4; ++w) h.vis[w] = vis[w];
          h.flags = cur.flags;
          h.g = cur.g;
          h.tok = cur.q.tok;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(HFULL + 8 * (i % kHdrs));
        const Tile t = cur;
        if (i + 1 < n) cur = walk.next(i + 1);
        ok = load(t, good, row, i == 0 ? 0 : 2 * i - 1);
        if (i == 0 && blockIdx.x == 0) write_tile_prefix(args, lane, held);  // (behind the first copies)
      }
    }
    if (!ok) {
      const uint64_t t0 = globaltimer();  // the copies already issued land before the CTA leaves
      while (globaltimer() - t0 < 100000ull) {
      }
    }
  } else if (warp >= 7) {
    // ------------------------------------------------------------ queries
    // A row's elements are all in the warp, 8 consecutive ones a lane and piece of 256.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int PC = D / 256;
    constexpr int HALF = NQ < 8 ? NQ : 8;  // rows in registers at a time
    bool ok = true;
    int32_t segs = 0;
    for (int32_t i = 0;; ++i) {
      const int hb = i % kHdrs;
      ok = __all_sync(0xffffffffu, mbar_wait_inline(HFULL + 8 * hb, (i / kHdrs) & 1, wc));
      if (!ok) break;
      const int32_t flags = hdrs[hb].flags, g = hdrs[hb].g, tok = hdrs[hb].tok;
      __syncwarp();
      if (lane == 0) mbar_arrive(HEMPTY + 8 * hb);
      if (flags & kEmpty) break;
      if (flags & kFirst) {
        const int qb = segs % C::NQB;
        unsigned char* const dst = gb + C::OFF_Q + qb * C::Q_BYTES;
        float* const qs = reinterpret_cast<float*>(gb + C::OFF_QS) + (segs % kQs) * 16;
        const __nv_bfloat16* const src = a.q + ((int64_t)tok * Hq + (int64_t)g * G) * D + 8 * lane;
        bool waited = false;
#pragma unroll 1
        for (int r0 = 0; ok && r0 < NQ; r0 += HALF) {
          uint4 x[HALF][PC];
#pragma unroll
          for (int k = 0; k < HALF; ++k) {
            const int row = r0 + k;
#pragma unroll
            for (int c = 0; c < PC; ++c)
              x[k][c] = row < G ? *reinterpret_cast<const uint4*>(src + (int64_t)row * D + 256 * c)
                                : make_uint4(0u, 0u, 0u, 0u);
          }
          if (!waited) {
            ok = __all_sync(0xffffffffu, mbar_wait(QEMPTY + 8 * qb, ((segs / C::NQB) & 1) ^ 1, wc));
            waited = true;
            if (!ok) break;
          }
#pragma unroll
          for (int k = 0; k < HALF; ++k) {
            const int row = r0 + k;
            if (row >= G) break;  // (uniform)
            float2 y[4 * PC];
#pragma unroll
            for (int c = 0; c < PC; ++c) {
              const uint32_t w[4] = {x[k][c].x, x[k][c].y, x[k][c].z, x[k][c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[4 * c + e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
            }
            const int32_t e = q8_exponent<32, 4 * PC>(y);
            const float inv = q8_pow2(-e);
#pragma unroll
            for (int c = 0; c < PC; ++c) {
              uint32_t hi[2], lo[2];
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                uint32_t h2[2], l2[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float2 v = y[4 * c + 2 * p + z];
                  const float2 s = make_float2(v.x * inv, v.y * inv);
                  h2[z] = e4m3x2(s);
                  const float2 got = q8_values(h2[z]);
                  l2[z] = e4m3x2(make_float2(16.f * (s.x - got.x), 16.f * (s.y - got.y)));
                }
                hi[p] = h2[0] | (h2[1] << 16);
                lo[p] = l2[0] | (l2[1] << 16);
              }
              // d = 256 c + 8 lane: its 128-d chunk, and 8 bytes of a swizzled row there
              const int d = 256 * c + 8 * lane;
              unsigned char* const at = dst + (d >> 7) * (C::QN * 128);
              const int pos = (((d & 127) >> 4) ^ (row & 7)) * 16 + (d & 8);
              *reinterpret_cast<uint2*>(at + row * 128 + pos) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(at + (NR + row) * 128 + pos) = make_uint2(lo[0], lo[1]);
            }
            if (lane == 0) qs[row] = q8_pow2(e) * a.sm_scale_log2;
          }
        }
        if (!ok) break;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(QFULL + 8 * qb);
          mbar_arrive(QSCALE + 8 * (segs % kQs));
        }
        ++segs;
      }
      if (flags & kEnd) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t IDESC_QK = idesc_e4m3(C::QN, false);
    constexpr uint32_t IDESC_PV = idesc_e4m3(C::PN, true);  // A (V) is MN-major
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
        ok = ok && wait1(SFREE + 8 * sb, ((i >> 1) & 1) ^ 1) && wait1(FULL(slot), round & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = sdesc(base + slot * C::SLOT, 16, NC * 1024);
        const uint64_t qd = sdesc(base + C::OFF_Q + ((segs - 1) % C::NQB) * C::Q_BYTES, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma8<IDESC_QK>(tmem + C::TM_S + sb * C::QN, kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                         qd + (uint64_t)(((kk >> 2) * (C::QN * 128) + (kk & 3) * 32) >> 4), kk > 0 ? 1u : 0u);
        commit1(EMPTY(slot));
        step();
        commit1(SFULL + 8 * sb);
        if (flags & kLast) commit1(QEMPTY + 8 * ((segs - 1) % C::NQB));
      }
      if (i > 0) {
        const int32_t jt = i - 1;
        const int pb = jt & 1, ob = pseg & 1;
        ok = wait1(PFULL + 8 * pb, (jt >> 1) & 1);
        if (ok && (pflags & kFirst)) ok = wait1(OFREE + 8 * ob, ((pseg >> 1) & 1) ^ 1);
        ok = ok && wait1(FULL(slot), round & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t pd = sdesc(base + C::OFF_P + pb * C::P_BYTES, 16, 1024);
#pragma unroll
        for (int mb = 0; mb < NC; ++mb) {  // 128 output columns: one chunk
          const uint64_t vd = sdesc(base + slot * C::SLOT + mb * 1024, 1024, NC * 1024);
#pragma unroll
          for (int kk = 0; kk < kT / 32; ++kk)  // 32 keys: four 8-key groups
            mma8<IDESC_PV>(tmem + C::TM_O + ob * C::O_COLS + mb * C::PN,
                           vd + (uint64_t)((kk * 4 * NC * 1024) >> 4), pd + (uint64_t)((kk * 32) >> 4),
                           ((pflags & kFirst) && kk == 0) ? 0u : 1u);
        }
        commit1(EMPTY(slot));
        step();
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
    float4* const fin = reinterpret_cast<float4*>(gb + C::OFF_FIN);
    const float* const qs0 = reinterpret_cast<const float*>(gb + C::OFF_QS);
    // l and its reference (of s), and P's reference (of s + v, less kTop)
    float l[NQ], ref[NQ], top[NQ];
    bool ok = true;
    int32_t segs = 0;
    struct Head {
      int32_t flags, g, tok;
      uint32_t mine, all, k, v;  // visible keys of the warp, of every warp; the key's scale bytes
    };
    // header of tile i, and the loads of this key's scales
    auto fetch = [&](int32_t i) {
      Head h{};
      const int hb = i % kHdrs;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(HFULL + 8 * hb, (i / kHdrs) & 1, wc));
      if (!ok) return h;
      const Q8Hdr& x = hdrs[hb];
      h.flags = x.flags;
      if (h.flags & kEmpty) return h;
      h.g = x.g;
      h.tok = x.tok;
      h.mine = x.vis[quarter];
      h.all = x.vis[0] & x.vis[1] & x.vis[2] & x.vis[3];
      if ((h.mine >> lane) & 1u) {
        const uint8_t* const at = qa.scales + x.row[row / kBox] + (row & (kBox - 1));
        h.k = *at;
        h.v = at[(int64_t)Hkv * ps];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(HEMPTY + 8 * hb);
      return h;
    };
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
      // O stands at P's reference, l at its own: the root of the factor between them, applied twice
      float inv[NQ], root[NQ];
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const float4 f = fin[x];
        inv[x] = f.x == 0.f ? 0.f : 1.f / f.x;
        root[x] = f.x == 0.f ? 0.f : ex2(0.5f * (f.z - f.y));
      }
#pragma unroll 1
      for (int p = 0; p < NC; ++p) {
        uint32_t o[C::PN];
        tmem_ld<C::PN>(tl + C::TM_O + (p_seg & 1) * C::O_COLS + p * C::PN, o);
        tmem_wait_ld();
        const int d = p * 128 + row;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          if (x >= G) break;
          const float sum = fmaf(__uint_as_float(o[2 * NR + x]), 1.f / 256,
                                 fmaf(__uint_as_float(o[NR + x]), 1.f / 16, __uint_as_float(o[x])));
          const float v = inv[x] == 0.f ? 0.f : sum * root[x] * inv[x] * root[x];
          if (p_flags & kSplit) args.rec_o[(rec + x) * D + d] = v;
          else a.out[(row0 + x) * D + d] = __float2bfloat16_rn(v);
        }
      }
      if (row < G) {
        const float4 f = fin[row];
        if (p_flags & kSplit) *reinterpret_cast<float2*>(args.rec_ml + (rec + row) * 2) = make_float2(f.y, f.x);
        else if (a.lse) a.lse[row0 + row] = f.x != 0.f ? (f.y + log2f(f.x)) * kLn2f : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(OFREE + 8 * (p_seg & 1));
    };
    Head h = fetch(0);
    for (int32_t i = 0;; ++i) {
      const int b = i & 1;
      if (any4(!ok)) break;  // all four warps leave together
      if (h.flags & kEmpty) break;
      Head next{};
      if (!(h.flags & kEnd)) next = fetch(i + 1);
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(SFULL + 8 * b, (i >> 1) & 1, wc));
      if (h.flags & kFirst) {
        // A place for scales is used again four segments on: by then the QK of a tile two past this
        // segment's last has run, and it waited for the last S to be read, which the scales are before.
        ok = ok && __all_sync(0xffffffffu, mbar_wait(QSCALE + 8 * (segs % kQs), (segs / kQs) & 1, wc));
        ++segs;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          l[x] = 0.f;
          ref[x] = top[x] = -INFINITY;
        }
      }
      const bool vis = (h.mine >> lane) & 1u;
      uint32_t sv[C::QN];
      tc_fence_after();
      tmem_ld<C::QN>(tl + C::TM_S + b * C::QN, sv);
      tmem_wait_ld();
      tc_fence_before();
      const float* const qs = qs0 + ((segs - 1) % kQs) * 16;
      float t[NQ];
      const float ks = q8_scale(h.k);
      const float ve = (float)((int32_t)h.v - 127);
      bool over = false;
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const float s = fmaf(__uint_as_float(sv[NR + x]), 1.f / 16, __uint_as_float(sv[x]));
        t[x] = vis ? s * ks * qs[x] : -INFINITY;
        over |= t[x] > ref[x] + kRescale || t[x] + ve > top[x] + (kTop + kRoom);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(SFREE + 8 * b);
      if (any4(over)) {
        // the rows' maxima over the tile, of s and of s + v, then references where they were outgrown
        float mine = -INFINITY, mine2 = -INFINITY;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          const float m = warp_max(t[x]), m2 = warp_max(t[x] + ve);
          if (lane == x) {
            mine = m;
            mine2 = m2;
          }
        }
        if (lane < NQ) {
          red[quarter * 16 + lane] = mine;
          red[64 + quarter * 16 + lane] = mine2;
        }
        sync4();
        float al[NQ];
        bool scaled = false;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          const float m = fmaxf(fmaxf(red[x], red[16 + x]), fmaxf(red[32 + x], red[48 + x]));
          const float m2 = fmaxf(fmaxf(red[64 + x], red[80 + x]), fmaxf(red[96 + x], red[112 + x]));
          if (m > ref[x] + kRescale) {
            const float to = m + kHeadroom;
            if (ref[x] != -INFINITY) {
              const float f = ex2(0.5f * (ref[x] - to));  // (its root, twice: attn_tc.cu)
              l[x] = (l[x] * f) * f;
            }
            ref[x] = to;
          }
          al[x] = 1.f;
          if (m2 > top[x] + (kTop + kRoom)) {
            const float to = m2 + kLead - kTop;
            if (top[x] != -INFINITY) {
              al[x] = ex2(0.5f * (top[x] - to));
              scaled = true;
            }
            top[x] = to;
          }
        }
        // O holds the segment's earlier tiles at the old references (uniform over the threads)
        if (scaled && !(h.flags & kFirst)) {
          const int32_t jt = i - 1;
          if (__all_sync(0xffffffffu, mbar_wait(PVDONE + 8 * (jt & 1), (jt >> 1) & 1, wc))) {
            tc_fence_after();
#pragma unroll 1
            for (int p = 0; p < NC; ++p) {
              uint32_t o[C::PN];
              const uint32_t at = tl + C::TM_O + ((segs - 1) & 1) * C::O_COLS + p * C::PN;
              tmem_ld<C::PN>(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int x = 0; x < NQ; ++x)
                  o[k * NR + x] = __float_as_uint((__uint_as_float(o[k * NR + x]) * al[x]) * al[x]);
              tmem_st<C::PN>(at, o);
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
      unsigned char* const pp = gb + C::OFF_P + b * C::P_BYTES + (row & 15);
#pragma unroll
      for (int x = 0; x < NQ; x += 2) {
        float2 w;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          if (x + z >= NQ) break;
          l[x + z] += ex2(t[x + z] - (ref[x + z] == -INFINITY ? 0.f : ref[x + z]));
          (z ? w.y : w.x) = ex2(t[x + z] + (ve - (top[x + z] == -INFINITY ? 0.f : top[x + z])));
        }
        const uint32_t p0 = e4m3x2(w);
        const float2 v0 = q8_values(p0);
        const float2 r1 = make_float2(16.f * (w.x - v0.x), 16.f * (w.y - v0.y));
        const uint32_t p1 = e4m3x2(r1);
        const float2 v1 = q8_values(p1);
        const uint32_t p2 = e4m3x2(make_float2(16.f * (r1.x - v1.x), 16.f * (r1.y - v1.y)));
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          if (x + z >= NQ) break;
          // row x of each term; the 16 keys of a piece are contiguous, pieces swizzled by the row
          unsigned char* const at = pp + (x + z) * 128 + (((row >> 4) ^ ((x + z) & 7)) << 4);
          at[0] = (unsigned char)(p0 >> (8 * z));
          at[NR * 128] = (unsigned char)(p1 >> (8 * z));
          at[2 * NR * 128] = (unsigned char)(p2 >> (8 * z));
        }
      }
      if (h.all != 0xFFFFFFFFu) {
        // V rows of keys that are not visible: zero once the copy has landed. The tile's V slot follows
        // K(i + 1) in the ring (the last tile's follows K(i)); the slot's use before was V(i - 2) or
        // earlier, which has been consumed (above), so a parity wait tells the phases apart.
        const int32_t at = (h.flags & kEnd) ? 2 * i + 1 : 2 * i + 2, sl = at % NS;
        ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(FULL(sl), (at / NS) & 1, wc));
        if (ok && !vis) {
          unsigned char* const v = gb + sl * C::SLOT + (row >> 3) * (NC * 1024) + (row & 7) * 128;
#pragma unroll
          for (int c = 0; c < 8 * NC; ++c)
            *reinterpret_cast<uint4*>(v + (c >> 3) * 1024 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
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
        if (lane < NQ) red[quarter * 16 + lane] = mine;
        sync4();
#pragma unroll
        for (int x = 0; x < NQ; ++x)
          if (row == x)
            fin[x] = make_float4((red[x] + red[16 + x]) + (red[32 + x] + red[48 + x]), ref[x], top[x], 0.f);
        sync4();
        pending = true;
        p_tile = i;
        p_flags = h.flags;
        p_g = h.g;
        p_tok = h.tok;
        p_seg = segs - 1;
      }
      if (h.flags & kEnd) break;
      h = next;
    }
    if (pending && ok) epilogue();
  }

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

template <int D, int NQ, int NR>
cudaError_t launch_q8(const AttnArgs& a, const Q8Dev& q8, cudaStream_t stream) {
  using C = Q8Cfg<D, NR>;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  const int32_t ps = a.pool.page_size, Hkv = a.pool.num_kv_heads;
  CUtensorMap tkv;
  {
    // (128 codes, row within an 8-row group, 128-d chunk, 8-row group): a box is 16 rows of a page
    const cuuint64_t rows = (cuuint64_t)a.pool.num_pages * 2 * Hkv * ps;
    cuuint64_t dims[4] = {128, 8, (cuuint64_t)C::NC, rows / 8};
    cuuint64_t strides[3] = {(cuuint64_t)D, 128, (cuuint64_t)D * 8};
    cuuint32_t box[4] = {128, 8, (cuuint32_t)C::NC, kBox / 8}, es[4] = {1, 1, 1, 1};
    if (enc(&tkv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, (void*)q8.codes, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  static PerDeviceOnce setup;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = setup.get(dev, [dev](int* n) {
    cudaError_t r = cudaFuncSetAttribute(q8_decode_kernel<D, NQ, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM);
    if (r != cudaSuccess) return r;
    return cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  }, &sms);
  if (e != cudaSuccess) return e;
  const int32_t S = std::max(1, std::min(std::min(sms, bounded_record_room(a, D)), a.max_tiles));
  Q8Args x;
  x.b.a = a;
  x.b.box_rows = kBox;
  x.b.box_lg = 31 - __builtin_clz((unsigned)kBox);
  x.b.page_lg = 31 - __builtin_clz((unsigned)ps);
  bounded_records(a, S, &x.b);
  x.scales = q8.scales;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, 1, 1);
  cfg.blockDim = dim3(kThreadsQ8, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, q8_decode_kernel<D, NQ, NR>, tkv, x);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_bounded_join(x.b, S, D, stream);
}

}  // namespace

bool q8_decode_supported(int32_t head_dim, int32_t group, int32_t page_size) {
  return (head_dim == 256 || head_dim == 512) && group >= 1 && group <= 16 && page_size >= kBox &&
         (page_size & (page_size - 1)) == 0;
}

cudaError_t launch_q8_decode(const AttnArgs& a, const Q8Dev& q8, int32_t head_dim, cudaStream_t stream) {
  if (a.plan.num_req == 0) return cudaSuccess;
  // the fewest softmax rows that hold the group
  if (head_dim == 256) {
    if (a.group <= 2) return launch_q8<256, 2, 8>(a, q8, stream);
    if (a.group <= 4) return launch_q8<256, 4, 8>(a, q8, stream);
    if (a.group <= 8) return launch_q8<256, 8, 8>(a, q8, stream);
    return launch_q8<256, 16, 16>(a, q8, stream);
  }
  if (a.group <= 4) return launch_q8<512, 4, 8>(a, q8, stream);
  if (a.group <= 8) return launch_q8<512, 8, 8>(a, q8, stream);
  return launch_q8<512, 16, 16>(a, q8, stream);
}

}  // namespace pg
