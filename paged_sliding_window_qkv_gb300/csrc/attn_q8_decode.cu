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
//   P = 2^(s + v - R) = p0 + p1 / 16 + p2 / 256 + p3 / 4096   v: of its V row; s in log2 units
//   O^T = V^T [p0 p1 p2 p3]^T  (M = 128 output columns, N = the rows four times, K = 32 keys a step)
// Two terms hold a bf16 query exactly (8 bits of significand) down to 2^-13 of the row's largest
// element; four hold a weight to 16 bits. The terms only widen N, which at these sizes costs nothing:
// an instruction's time is that of reading A (the codes) from shared memory.
//
// e4m3 reaches from 2^-9 to 448, so R must stand near the row's largest s + v, not 2^48 off as in the
// bf16 kernels: it moves when an exponent outgrows it, to leave kLead + kRoom octaves of room. A weight's
// last term ends 2^-22 below 1, 2^-26 below the largest: n keys there are off by n times that together, a
// bf16 output's half step for n = 131072. (With three terms, and 2^-22 below the largest, 16384 such keys lost
// 0.4% of the output.) The row sum keeps its own reference (of s alone) and adds the unrounded weights.
//
// Work, walk, records and join are those of attn_bounded_decode.cu; a ring slot is a tile of K or V
// (128 keys x head_dim codes: three slots of 64 KB, or six of 32 KB), in the order K0 K1 V0 K2 V1 ...
//   warps 0, 6  producers of K (with a header a tile) and of V: one 4-D box per 16 keys
//   warp 7      the group's query rows into their terms, a segment ahead as far as their buffer allows
//   (the last)  (groups above 4: four warps, which share the rows); and V rows of keys that are not visible
//               to zero, whatever they held, once a tile's weights and V have arrived
//   warp 1      MMA issuer: QK of tile i + 1 before PV of tile i
//   warps 2-5   softmax: a thread is a key and up to 8 query rows; its row scales load a tile ahead.
//   (8-11)      Groups above 8 take two such sets, which share nothing but the tiles. (One set over
//               16 rows took some 5,000 cycles a tile, as long as the tile's bytes; and references
//               found by a reduction a row 9,000 where they moved: 146 us on the 64 requests below.)
// Measured: 64 requests of up to 16384 keys at head_dim 512, 16 heads, 101 us (5.8 TB/s over the call; the read-back and
// the bf16 kernel take 450); 64 under a window of 1023 at head_dim 256, 16 / 8 heads, 50 us (317); one of 8001
// keys at head_dim 512 16.5 us (latency of two launches). Bound by HBM, and by CTAs that end unevenly.
// Every wait is bounded, as there.
#include "bounded_decode.cuh"
#include "q8.cuh"

#include <math.h>

#include <algorithm>

namespace pg {
namespace {

constexpr int kQ8Ctas = 320;  // records are sized for at most this many CTAs (two an SM)
constexpr int kFix = 64;  // a tile flag: it has keys that are not visible, so V waits to be cleared
constexpr int kQs = 4;  // segments whose query scales are kept
constexpr int kBox = 16, kBoxes = kT / kBox;  // key rows of a box, boxes of a tile
// P is at most 448 where a weight stands kRoom octaves above its reference; a reference is set kLead
// above the largest weight (P = 2^(8 - kLead) there).
constexpr float kTop = 8.f, kLead = 4.f, kRoom = 0.8f;
constexpr int kTerms = 4;  // of a weight

struct alignas(16) Q8Hdr {
  uint32_t vis[4];       // visible keys
  int32_t row[kBoxes];   // each box's first K row of the layer (-1: not loaded)
  int32_t flags, g, tok;
};

// NQ: query rows of the softmax; NR: rows of a term (8 or 16, the group padded)
template <int D, int NQ, int NR>
struct Q8Cfg {
  static constexpr int SETS = NQ > 8 ? 2 : 1;   // sets of four softmax warps
  static constexpr int CQ = NQ / SETS;          // query rows of a set
  static constexpr int QW = NQ > 4 ? 4 : 1;     // query warps
  static constexpr int THREADS = 224 + 32 * QW + 128 * (SETS - 1);
  // Small groups at head_dim 256: two CTAs an SM, each with half the ring, so that one streams while the
  // other starts or ends a segment (of some 9 tiles under a window of 1023).
  static constexpr int PER_SM = D == 256 && NQ <= 4 ? 2 : 1;
  static constexpr int NC = D / 128;            // 128-d chunks of a row
  static constexpr int SLOT = kT * D;
  static constexpr int NSLOT = D == 256 ? 6 / PER_SM : 3;
  static constexpr int QN = 2 * NR;             // columns of S: two terms
  static constexpr int PN = kTerms * NR;        // of O
  // O buffers (segments): two, but where tensor memory holds one beside the scores
  static constexpr int NOB = D == 512 && NR == 16 ? 1 : 2;
  static constexpr int NQB = D == 256 && PER_SM == 1 ? 2 : 1;  // query buffers (segments)
  static constexpr int Q_BYTES = NC * QN * 128; // [128-d chunk][QN rows][128 B]
  static constexpr int P_BYTES = PN * 128;      // [PN rows][128 keys]
  static constexpr int OFF_Q = NSLOT * SLOT;
  static constexpr int OFF_P = OFF_Q + NQB * Q_BYTES;
  static constexpr int OFF_QS = OFF_P + 2 * P_BYTES;                 // [kQs][16] query scales
  static constexpr int OFF_HDR = OFF_QS + kQs * 16 * 4;
  static constexpr int OFF_RED = OFF_HDR + kHdrs * (int)sizeof(Q8Hdr);  // [sets][4 warps][8] pairs
  static constexpr int OFF_FIN = OFF_RED + SETS * 4 * 8 * 8;         // [16] (l, its reference, P's)
  static constexpr int OFF_BAR = OFF_FIN + 16 * 16;
  // FULL, EMPTY; QFULL[2], QEMPTY[2], HFULL[4], HEMPTY[4], SFULL[2], SFREE[2], PFULL[2], PVDONE[2],
  // OFREE[2], DRAIN, QSCALE[4], VREADY[2], VCLEAR[2]
  static constexpr int NBAR = 2 * NSLOT + 4 + 8 + 10 + 1 + kQs + 4;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static constexpr uint32_t TM_O = 0, O_COLS = NC * PN, TM_S = NOB * O_COLS;
  static constexpr uint32_t TM_COLS = TM_S + 2 * QN <= 256 ? 256 : 512;
  static_assert(PER_SM * (SMEM + 1024) <= 228 * 1024, "shared memory");
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
// Whether the phase of the given parity is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// two e4m3 numbers, the first in the low byte, and what they stand for
__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t e4m3x2(__half2 v) {
  const __half2_raw r = *reinterpret_cast<const __half2_raw*>(&v);
  return __nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3);  // (without saturation it takes a subroutine)
}
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

template <int D, int NQ, int NR>
__global__ void __launch_bounds__(Q8Cfg<D, NQ, NR>::THREADS, Q8Cfg<D, NQ, NR>::PER_SM)
q8_decode_kernel(const __grid_constant__ CUtensorMap tm_kv, Q8Args qa) {
  using C = Q8Cfg<D, NQ, NR>;
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
                 OFREE = SFULL + 64, DRAIN = SFULL + 80, QSCALE = SFULL + 88, VREADY = QSCALE + 8 * kQs,
                 VCLEAR = VREADY + 16;
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
      mbar_init(QFULL + 8 * b, C::QW);
      mbar_init(QEMPTY + 8 * b, 1);
      mbar_init(SFULL + 8 * b, 1);
      mbar_init(SFREE + 8 * b, 4 * C::SETS);
      mbar_init(PFULL + 8 * b, 4 * C::SETS);
      mbar_init(PVDONE + 8 * b, 1);
      mbar_init(OFREE + 8 * b, 4 * C::SETS);
    }
    for (int h = 0; h < kHdrs; ++h) {
      mbar_init(HFULL + 8 * h, 1);
      mbar_init(HEMPTY + 8 * h, 4 * C::SETS + 1 + C::QW);  // the softmax warps, the query warps and the MMA issuer
    }
    for (int q = 0; q < kQs; ++q) mbar_init(QSCALE + 8 * q, C::QW);
    for (int q = 0; q < 2; ++q) {
      mbar_init(VREADY + 8 * q, 1);
      mbar_init(VCLEAR + 8 * q, 4 * C::SETS);
    }
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
    __syncwarp();  // (lane 0 has set up the barriers)
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
      wait_previous(a);
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
      wait_previous(a);
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
          h.flags = cur.flags | ((vis[0] & vis[1] & vis[2] & vis[3]) == 0xFFFFFFFFu ? 0 : kFix);
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
  } else if (warp == 7 || (C::QW > 1 && warp > C::THREADS / 32 - C::QW)) {
    // ------------------------------------------------------------ queries
    // A row's elements are all in the warp, 8 consecutive ones a lane and piece of 256.
    wait_previous(a);
    constexpr int PC = D / 256, ROWS = NQ / C::QW;  // (NQ is 2, 4, 8 or 16)
    const int first = warp == 7 ? 0 : C::THREADS / 32 - warp;
    int32_t segs = 0, i = 0, j = 0;  // headers read, and given back
    int32_t g = 0, tok = 0, fixes = 0;
    bool end = false, fresh = false;  // fresh: the last header read began a segment whose queries are to come
    uint64_t since = 0;               // when nothing was left to do
    // Headers are read as they come, for the queries of new segments, and given back; by warp 7 once its tile's
    // V rows need nothing more. Nothing here waits for one thing alone: the query buffer may come free
    // only behind a tile whose V rows are still to be cleared.
    while (!end || fresh || j < i) {
      bool idle = true;
      if (!end && !fresh && i - j < kHdrs &&
          __all_sync(0xffffffffu, mbar_test(HFULL + 8 * (i % kHdrs), (i / kHdrs) & 1))) {
        idle = false;
        const Q8Hdr& h = hdrs[i % kHdrs];
        ++i;
        if (h.flags & kEmpty) break;
        end = h.flags & kEnd;
        fresh = h.flags & kFirst;
        g = h.g;
        tok = h.tok;
      }
      if (fresh) {
        const int qb = segs % C::NQB;
        if (__all_sync(0xffffffffu, mbar_test(QEMPTY + 8 * qb, ((segs / C::NQB) & 1) ^ 1))) {
          idle = fresh = false;
          unsigned char* const dst = gb + C::OFF_Q + qb * C::Q_BYTES;
          float* const qs = reinterpret_cast<float*>(gb + C::OFF_QS) + (segs % kQs) * 16;
          const __nv_bfloat16* const src = a.q + ((int64_t)tok * Hq + (int64_t)g * G) * D + 8 * lane;
          // A loop of few instructions over the rows, two at a time (unrolled over all of them it took
          // 10,000 cycles at a CTA's start, most of it to fetch the code)
          constexpr int STEP = ROWS < 2 ? 1 : 2;
          uint4 x[STEP][PC];
          auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < STEP; ++k)
#pragma unroll
              for (int c = 0; c < PC; ++c) {
                const int row = first + C::QW * (k0 + k);
                x[k][c] = row < G ? *reinterpret_cast<const uint4*>(src + (int64_t)row * D + 256 * c)
                                  : make_uint4(0u, 0u, 0u, 0u);
              }
          };
          load(0);
#pragma unroll 1
          for (int k0 = 0; k0 < ROWS; k0 += STEP) {
            uint4 y[STEP][PC];
#pragma unroll
            for (int k = 0; k < STEP; ++k)
#pragma unroll
              for (int c = 0; c < PC; ++c) y[k][c] = x[k][c];
            if (k0 + STEP < ROWS) load(k0 + STEP);
            float f[STEP];
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
              __nv_bfloat162 m = __habs2(as_bf2(y[k][0].x));
#pragma unroll
              for (int c = 0; c < PC; ++c) {
                if (c > 0) m = __hmax2(m, __habs2(as_bf2(y[k][c].x)));
                m = __hmax2(m, __habs2(as_bf2(y[k][c].y)));
                m = __hmax2(m, __habs2(as_bf2(y[k][c].z)));
                m = __hmax2(m, __habs2(as_bf2(y[k][c].w)));
              }
              f[k] = fmaxf(__low2float(m), __high2float(m));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
              for (int k = 0; k < STEP; ++k) f[k] = fmaxf(f[k], __shfl_xor_sync(0xffffffffu, f[k], o));
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
              const int row = first + C::QW * (k0 + k);
              const int32_t e = q8_exponent_of(f[k] > 0.f ? f[k] : 0.f);
              const float inv = q8_pow2(-e);
#pragma unroll
              for (int c = 0; c < PC; ++c) {
                const uint32_t w[4] = {y[k][c].x, y[k][c].y, y[k][c].z, y[k][c].w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                  // (16 bits hold 8 of significand down to 2^-17, and 2^-25 below: finer than a1 / 16)
                  const __half2 s = __floats2half2_rn(__uint_as_float(w[p] << 16) * inv,
                                                      __uint_as_float(w[p] & 0xFFFF0000u) * inv);
                  hi[p] = e4m3x2(s);
                  lo[p] = e4m3x2(__hmul2(__hsub2(s, q8_halves(hi[p])), __float2half2_rn(16.f)));
                }
                // d = 256 c + 8 lane: its 128-d chunk, and 8 bytes of a swizzled row there
                const int d = 256 * c + 8 * lane;
                unsigned char* const at = dst + (d >> 7) * (C::QN * 128);
                const int pos = (((d & 127) >> 4) ^ (row & 7)) * 16 + (d & 8);
                *reinterpret_cast<uint2*>(at + row * 128 + pos) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                *reinterpret_cast<uint2*>(at + (NR + row) * 128 + pos) =
                    make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
              }
              // (NaN is passed over by the maxima and stays NaN in the terms; the conversion turns an
              // infinity into 448, so its row's scores become NaN here)
              if (lane == 0) qs[row] = row >= G ? 0.f : f[k] == INFINITY ? NAN : q8_pow2(e) * a.sm_scale_log2;
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(QFULL + 8 * qb);
            mbar_arrive(QSCALE + 8 * (segs % kQs));
          }
          ++segs;
        }
      }
      if (j < i) {
        const int hb = j % kHdrs;
        const Q8Hdr& h = hdrs[hb];
        // Warp 7 clears a tile's V rows once its weights have been written: its scores have then been read and
        // PV of the tile two before is done, so the V slot's use before (K(j), V(j - 2) or an earlier one; V(j)
        // follows K(j + 1) in the ring, the last one K(j)) has been consumed too. The weights of such tiles
        // have barriers of their own (VCLEAR). A parity test takes two phases for none, and the weights of tiles
        // without hidden keys wait for nothing of this warp: on PFULL two of them could pass while queries are
        // converted here. Those of a third such tile wait for the first one's PV, which waits for VREADY.
        const bool fix = warp == 7 && (h.flags & kFix);
        bool done = !fix;
        if (fix && __all_sync(0xffffffffu, mbar_test(VCLEAR + 8 * (fixes & 1), (fixes >> 1) & 1))) {
          const int32_t at = (h.flags & kEnd) ? 2 * j + 1 : 2 * j + 2, sl = at % NS;
          done = __all_sync(0xffffffffu, mbar_test(FULL(sl), (at / NS) & 1));
          if (done) {
            // eight lanes a row
#pragma unroll 1
            for (int k = lane >> 3; k < kT; k += 4) {
              if ((h.vis[k >> 5] >> (k & 31)) & 1u) continue;
              unsigned char* const v = gb + sl * C::SLOT + (k >> 3) * (NC * 1024) + (k & 7) * 128 + (lane & 7) * 16;
#pragma unroll
              for (int c = 0; c < NC; ++c) *reinterpret_cast<uint4*>(v + c * 1024) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
          }
        }
        if (done) {
          idle = false;
          __syncwarp();
          if (lane == 0) {
            if (fix) mbar_arrive(VREADY + 8 * (fixes & 1));
            mbar_arrive(HEMPTY + 8 * hb);
          }
          fixes += fix ? 1 : 0;
          ++j;
        }
      }
      if (!idle) {
        since = 0;
        continue;
      }
      const uint64_t now = globaltimer();
      if (since == 0) since = now;
      if (__any_sync(0xffffffffu, *abort_flag != 0 || now - since > wc.limit_ns)) {
        if (lane == 0 && *abort_flag == 0) {
          atomicOr(a.status, kStatusTimeout);
          *abort_flag = 1;
        }
        break;
      }
      // (the softmax warps want the issue slots: a spinning warp here cost 3% of a step)
      if (j == i && !fresh) mbar_try_wait(HFULL + 8 * (i % kHdrs), (i / kHdrs) & 1);
      else __nanosleep(100);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t IDESC_QK = idesc_e4m3(C::QN, false);
    constexpr uint32_t IDESC_PV = idesc_e4m3(C::PN, true);  // A (V) is MN-major
    auto wait1 = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, wc));
    };
    int slot = 0, round = 0;
    auto step = [&]() {
      if (++slot == NS) { slot = 0; ++round; }
    };
    int32_t segs = 0, flags = 0, pflags = 0, pseg = 0, fixes = 0;
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
        const int pb = jt & 1, ob = pseg % C::NOB;
        ok = wait1(PFULL + 8 * pb, (jt >> 1) & 1);
        if (ok && (pflags & kFirst)) ok = wait1(OFREE + 8 * ob, ((pseg / C::NOB) & 1) ^ 1);
        ok = ok && wait1(FULL(slot), round & 1);
        if (ok && (pflags & kFix)) {
          ok = wait1(VREADY + 8 * (fixes & 1), (fixes >> 1) & 1);
          ++fixes;
        }
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
    wait_previous(a);
    constexpr int CQ = C::CQ;
    const int set = warp >= 8 ? 1 : 0, bar = 1 + set;
    const int x0 = set * CQ;  // the set's first query row
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // the thread's key of each tile, and output column of 128
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + x0;
    float2* const red = reinterpret_cast<float2*>(gb + C::OFF_RED) + set * 32;
    float4* const fin = reinterpret_cast<float4*>(gb + C::OFF_FIN) + x0;
    const float* const qs0 = reinterpret_cast<const float*>(gb + C::OFF_QS) + x0;
    const int32_t Gs = min(max(G - x0, 0), CQ);  // rows of the group in the set
    // l and its reference (of s), and P's reference (of s + v, less kTop)
    float l[CQ], ref[CQ], top[CQ];
    float my_ref = -INFINITY, my_top = -INFINITY;  // those of row set_col(lane)
    bool ok = true;
    int32_t segs = 0, fixes = 0;
    struct Head {
      int32_t flags, g, tok;
      uint32_t mine, k, v;  // visible keys of the warp; the key's scale bytes
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
      const int64_t row0 = (int64_t)p_tok * Hq + (int64_t)p_g * G + x0;
      const int64_t rec = ((int64_t)blockIdx.x * 2 + ((p_flags & kRec1) ? 1 : 0)) * G + x0;
      // O stands at P's reference, l at its own: the root of the factor between them, applied twice
      float inv[CQ], root[CQ];
#pragma unroll
      for (int x = 0; x < CQ; ++x) {
        const float4 f = fin[x];
        inv[x] = f.x == 0.f ? 0.f : 1.f / f.x;
        root[x] = f.x == 0.f ? 0.f : ex2(0.5f * (f.z - f.y));
      }
#pragma unroll 1
      for (int p = 0; p < NC; ++p) {
        uint32_t o[kTerms][8];
        __syncwarp();
        const uint32_t at = tl + C::TM_O + (p_seg % C::NOB) * C::O_COLS + p * C::PN;
#pragma unroll
        for (int k = 0; k < kTerms; ++k) tmem_ld8(at + k * NR, o[k]);
        tmem_wait_ld();
        const int d = p * 128 + row;
#pragma unroll
        for (int x = 0; x < CQ; ++x) {
          if (x >= Gs) break;
          float sum = __uint_as_float(o[kTerms - 1][x]);
#pragma unroll
          for (int k = kTerms - 2; k >= 0; --k) sum = fmaf(sum, 1.f / 16, __uint_as_float(o[k][x]));
          const float v = inv[x] == 0.f ? 0.f : sum * root[x] * inv[x] * root[x];
          if (p_flags & kSplit) args.rec_o[(rec + x) * D + d] = v;
          else a.out[(row0 + x) * D + d] = __float2bfloat16_rn(v);
        }
      }
      if (row < Gs) {
        const float4 f = fin[row];
        if (p_flags & kSplit) *reinterpret_cast<float2*>(args.rec_ml + (rec + row) * 2) = make_float2(f.y, f.x);
        else if (a.lse) a.lse[row0 + row] = f.x != 0.f ? (f.y + log2f(f.x)) * kLn2f : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(OFREE + 8 * (p_seg % C::NOB));
    };
    Head h = fetch(0);
    const bool none = any_of(bar, !ok) || (h.flags & kEmpty);  // (all of the set's warps leave together)
    for (int32_t i = 0; !none; ++i) {
      const int b = i & 1;
      Head next{};
      if (!(h.flags & kEnd)) next = fetch(i + 1);
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(SFULL + 8 * b, (i >> 1) & 1, wc));
      if (h.flags & kFirst) {
        // A place for scales is used again four segments on: by then the QK of a tile two past this
        // segment's last has run, and it waited for the last S to be read, which the scales are before.
        ok = ok && __all_sync(0xffffffffu, mbar_wait(QSCALE + 8 * (segs % kQs), (segs / kQs) & 1, wc));
        ++segs;
#pragma unroll
        for (int x = 0; x < CQ; ++x) {
          l[x] = 0.f;
          ref[x] = top[x] = -INFINITY;
        }
        my_ref = my_top = -INFINITY;
      }
      const bool vis = (h.mine >> lane) & 1u;
      uint32_t s0[8], s1[8];
      tc_fence_after();
      __syncwarp();  // (a tensor-memory access is the whole warp's: it meets behind the lanes' waits)
      tmem_ld8(tl + C::TM_S + b * C::QN, s0);
      tmem_ld8(tl + C::TM_S + b * C::QN + NR, s1);
      tmem_wait_ld();
      tc_fence_before();
      const float* const qs = qs0 + ((segs - 1) % kQs) * 16;
      float t[CQ];
      const float ks = q8_scale(h.k);
      const float ve = h.v == 255u ? NAN : (float)((int32_t)h.v - 127);
      bool over = false;
#pragma unroll
      for (int x = 0; x < CQ; ++x) {
        const float s = fmaf(__uint_as_float(s1[x]), 1.f / 16, __uint_as_float(s0[x]));
        t[x] = vis ? s * ks * qs[x] : -INFINITY;
        over |= t[x] > ref[x] + kRescale || t[x] + ve > top[x] + (kTop + kRoom);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(SFREE + 8 * b);
      if ((h.flags & kFirst) || any_of(bar, over || !ok)) {
        if (any_of(bar, !ok)) break;
        // The rows' maxima over the tile, of s and of s + v, then references where they were outgrown:
        // lane i looks after row set_col(i), and every lane takes what it finds.
        float u[CQ];
#pragma unroll
        for (int x = 0; x < CQ; ++x) u[x] = t[x] + ve;
        const int col = set_col<CQ>(lane);
        const float2 mine = make_float2(warp_reduce<CQ, false>(t, lane), warp_reduce<CQ, false>(u, lane));
        if (lane % (32 / CQ) == 0) red[quarter * 8 + col] = mine;
        sync_set(bar);
        float2 m = red[col];
#pragma unroll
        for (int k = 1; k < 4; ++k) {
          const float2 y = red[8 * k + col];
          m = make_float2(fmaxf(m.x, y.x), fmaxf(m.y, y.y));
        }
        const bool move_l = m.x > my_ref + kRescale, move_o = m.y > my_top + (kTop + kRoom);
        const float to_l = move_l ? m.x + kHeadroom : my_ref, to_o = move_o ? m.y + kLead - kTop : my_top;
        // roots of the factors, to be applied twice (attn_tc.cu)
        const float fl = move_l && my_ref != -INFINITY ? ex2(0.5f * (my_ref - to_l)) : 1.f;
        const float fo = move_o && my_top != -INFINITY ? ex2(0.5f * (my_top - to_o)) : 1.f;
        const bool scaled = __any_sync(0xffffffffu, move_o && my_top != -INFINITY);
        my_ref = to_l;
        my_top = to_o;
        float al[CQ];
#pragma unroll
        for (int x = 0; x < CQ; ++x) {
          const int from = x * (32 / CQ);
          ref[x] = __shfl_sync(0xffffffffu, my_ref, from);
          top[x] = __shfl_sync(0xffffffffu, my_top, from);
          al[x] = __shfl_sync(0xffffffffu, fo, from);
          const float f = __shfl_sync(0xffffffffu, fl, from);
          l[x] = (l[x] * f) * f;
        }
        // O holds the segment's earlier tiles at the old references (uniform over the set)
        if (scaled && !(h.flags & kFirst)) {
          const int32_t jt = i - 1;
          if (__all_sync(0xffffffffu, mbar_wait(PVDONE + 8 * (jt & 1), (jt >> 1) & 1, wc))) {
            tc_fence_after();
            __syncwarp();
#pragma unroll 1
            for (int p = 0; p < NC; ++p) {
              uint32_t o[kTerms][8];
              const uint32_t at = tl + C::TM_O + ((segs - 1) % C::NOB) * C::O_COLS + p * C::PN;
#pragma unroll
              for (int k = 0; k < kTerms; ++k) tmem_ld8(at + k * NR, o[k]);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < kTerms; ++k) {
#pragma unroll
                for (int x = 0; x < CQ; ++x) o[k][x] = __float_as_uint((__uint_as_float(o[k][x]) * al[x]) * al[x]);
                tmem_st8(at + k * NR, o[k]);
              }
            }
            tmem_wait_st();
          } else {
            ok = false;
          }
        }
        sync_set(bar);  // red has been read
      }
      // the P buffer is free once PV(i - 2) has read it
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(PVDONE + 8 * b, ((i >> 1) & 1) ^ 1, wc));
      unsigned char* const pp = gb + C::OFF_P + b * C::P_BYTES + (row & 15);
#pragma unroll
      for (int x = 0; x < CQ; x += 2) {
        float2 w;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          l[x + z] += ex2(t[x + z] - (ref[x + z] == -INFINITY ? 0.f : ref[x + z]));
          (z ? w.y : w.x) = ex2(t[x + z] + (ve - (top[x + z] == -INFINITY ? 0.f : top[x + z])));
        }
        uint32_t p[kTerms];
#pragma unroll
        for (int k = 0; k < kTerms; ++k) {
          p[k] = e4m3x2(w);
          const float2 v = q8_values(p[k]);
          w = make_float2(16.f * (w.x - v.x), 16.f * (w.y - v.y));
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          // row x of each term; the 16 keys of a piece are contiguous, pieces swizzled by the row
          unsigned char* const at = pp + (x0 + x + z) * 128 + (((row >> 4) ^ ((x + z) & 7)) << 4);
#pragma unroll
          for (int k = 0; k < kTerms; ++k) at[k * NR * 128] = (unsigned char)(p[k] >> (8 * z));
        }
      }
      fence_proxy_async();  // the MMA reads P through the async proxy
      tc_fence_before();    // and O after any rescaling above
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(PFULL + 8 * b);
        if (h.flags & kFix) mbar_arrive(VCLEAR + 8 * (fixes & 1));
      }
      fixes += h.flags & kFix ? 1 : 0;
      if (pending && ok) epilogue();
      pending = false;
      if (h.flags & kLast) {
        // the row sums over the 128 keys of every tile, and the references, for the epilogue
        const int col = set_col<CQ>(lane);
        const float mine = warp_reduce<CQ, true>(l, lane);
        if (lane % (32 / CQ) == 0) red[quarter * 8 + col].x = mine;
        sync_set(bar);
#pragma unroll
        for (int x = 0; x < CQ; ++x)
          if (row == x) fin[x] = make_float4((red[x].x + red[8 + x].x) + (red[16 + x].x + red[24 + x].x), ref[x], top[x], 0.f);
        sync_set(bar);
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
  wait_beside(a);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(DRAIN, 0)) {
      if (globaltimer() - t0 > a.wait_ns) {
        atomicOr(a.status, kStatusTimeout);
        break;
      }
    }
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TM_COLS) : "memory");
  }
}

template <int D, int NQ, int NR>
cudaError_t launch_q8(const AttnArgs& a, const Q8Dev& q8, cudaStream_t stream) {
  using C = Q8Cfg<D, NQ, NR>;
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
  const int32_t S = std::max(1, std::min(std::min((a.beside > 0 ? std::min(a.beside, sms) : sms) * C::PER_SM, bounded_record_room(a, D, kQ8Ctas)), a.max_tiles));
  Q8Args x;
  x.b.a = a;
  x.b.box_rows = kBox;
  x.b.box_lg = 31 - __builtin_clz((unsigned)kBox);
  x.b.page_lg = 31 - __builtin_clz((unsigned)ps);
  bounded_records(a, S, &x.b);
  x.scales = q8.scales;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
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

size_t q8_decode_ws_bytes(int32_t num_req, int32_t group, int32_t head_dim, int32_t max_tiles) {
  return bounded_records_bytes(num_req, group, head_dim, std::min(kQ8Ctas, max_tiles));
}

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
