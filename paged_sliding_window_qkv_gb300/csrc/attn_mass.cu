// Accumulated attention weights of a paged cache ("feat(gemma4): paged KV serving across both
// attention families", Description: the global layers attend to every key, so their cache is the
// one that grows without bound; the weights decide which of its keys an eviction gives up).
//
// For a step's rows t, the heads h of KV head g and a key j:
//   mass[g][j] (+)= sum_{t, h} exp(scale <q_th, k_j> - lse_th)
// over the rows that see j. Keys the step itself wrote (j >= start_pos) start from zero and get
// their position recorded; older keys add. The normaliser lse of a row is known only after all of
// its keys, so the sums are a second pass behind the attention:
//   decode   the attention kernel keeps the step's scores (Hq floats per key, against the
//            2 Hkv D bf16 of its K and V rows), and one thread per key adds the group's weights;
//   prefill  the scores are formed again with keys as MMA rows, S^T = K Q^T: a key's sum then
//            runs along its own row, in registers, with no atomics and in one fixed order.
#include "mass.cuh"
#include "pg_internal.h"

#include <cuda_bf16.h>
#include <math.h>

#include <mutex>

namespace pg {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^x with the hardware exponential (-inf gives 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int D>
__device__ __forceinline__ uint32_t swz(int m, int c) {
  return (uint32_t)(m * (D * 2) + ((c ^ (m & 7)) << 4));
}

// Decode: one thread per key adds the weights of its query heads from the kept scores.
constexpr int kDecThreads = 256;
__global__ void __launch_bounds__(kDecThreads) mass_decode_kernel(MassArgs m, int32_t blocks_per_req) {
  const AttnArgs& a = m.attn;
  extern __shared__ float s_lse[];  // the request's lse, log2 units
  const int32_t r = (int32_t)blockIdx.x / blocks_per_req;
  const int32_t ps = a.pool.page_size, Hq = a.num_qo_heads, G = a.group;
  const MassReq q = mass_req(a.plan, r, ps);
  for (int h = threadIdx.x; h < Hq; h += kDecThreads) s_lse[h] = a.lse[(int64_t)q.q0 * Hq + h] * kLog2e;
  __syncthreads();
  const int32_t p = q.sp;
  // (a graph's plan may have grown since the capture: the blocks stride over the keys)
  for (int64_t i = (int32_t)blockIdx.x % blocks_per_req * kDecThreads + (int32_t)threadIdx.x; i < q.n;
       i += (int64_t)blocks_per_req * kDecThreads) {
    const int32_t rel = (int32_t)i, j = q.ks0 + rel;
    if (j > p || !(a.window_left < 0 || p - j <= a.window_left || j < a.num_sink)) continue;
    const int64_t slot = (int64_t)q.kvp0 * ps + rel;
    const int32_t page = mass_page(a.plan, q, rel, ps, a.pool.num_pages);
    if (page == a.pool.num_pages || slot >= a.logit_slots) {
      atomicOr(a.status, kStatusBounds);
      continue;
    }
    const float* s = a.logits + slot * Hq;
    for (int32_t g = 0; g < a.pool.num_kv_heads; ++g) {
      float sum = 0.f;
      for (int32_t h = g * G; h < (g + 1) * G; ++h) sum += ex2(s[h] - s_lse[h]);
      mass_store(a, q, page, g, rel, sum);
    }
  }
}

// Prefill, any page size: one CTA per (request, KV head, 64 keys), four warps of 16 keys each;
// the keys stay in shared memory while the query rows that see them pass by 32 at a time. (A graph's
// plan may have grown since the capture: a request's CTAs stride over its keys.)
constexpr int kKeys = 64, kRows = 32, kMassThreads = 128;
template <int D>
__global__ void __launch_bounds__(kMassThreads) mass_prefill_kernel(MassArgs m, int32_t tiles_per_req) {
  const AttnArgs& a = m.attn;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* sK = smem;
  unsigned char* sQ = sK + kKeys * D * 2;
  float* sL = reinterpret_cast<float*>(sQ + kRows * D * 2);  // lse of the 32 rows, log2 units
  constexpr int CH = D / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t Hkv = a.pool.num_kv_heads, ps = a.pool.page_size, G = a.group, Hq = a.num_qo_heads;
  const int32_t g = (int32_t)blockIdx.x % Hkv;
  const int32_t kt = ((int32_t)blockIdx.x / Hkv) % tiles_per_req;
  const int32_t r = (int32_t)blockIdx.x / Hkv / tiles_per_req;
  const MassReq q = mass_req(a.plan, r, ps);
  const int32_t W = a.window_left;
  const int gid = lane >> 2, tig = lane & 3;
  for (int64_t first = (int64_t)kt * kKeys; first < q.n; first += (int64_t)tiles_per_req * kKeys) {
    const int32_t rel0 = (int32_t)first;
    __syncthreads();  // the previous keys have been read
    const int32_t k0 = q.ks0 + rel0, nk = min(kKeys, q.n - rel0);
    // K rows; rows of no key, or on a page that is out of range, are zero
    for (int idx = tid; idx < kKeys * CH; idx += kMassThreads) {
      const int k = idx / CH, c = idx % CH;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (k < nk) {
        const int32_t page = mass_page(a.plan, q, rel0 + k, ps, a.pool.num_pages);
        if (page < a.pool.num_pages)
          v = *reinterpret_cast<const uint4*>(a.pool.layer_base + (int64_t)page * a.pool.stride_page +
                                              (int64_t)g * a.pool.stride_head +
                                              (int64_t)((rel0 + k) % ps) * D + c * 8);
      }
      *reinterpret_cast<uint4*>(sK + swz<D>(k, c)) = v;
    }
    // the tokens that may see a key of the tile
    const int32_t t0 = max(0, k0 - q.sp);
    int64_t t1 = q.len;
    if (W >= 0 && k0 >= a.num_sink) t1 = min(t1, (int64_t)k0 + nk - 1 + W - q.sp + 1);
    const int64_t row_end = t1 * G;
    float sum[2] = {0.f, 0.f};
    for (int64_t row0 = (int64_t)t0 * G; row0 < row_end; row0 += kRows) {
      __syncthreads();  // the previous rows have been read
      for (int idx = tid; idx < kRows * CH; idx += kMassThreads) {
        const int n = idx / CH, c = idx % CH;
        const int64_t row = row0 + n;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < row_end)
          v = *reinterpret_cast<const uint4*>(
              a.q + ((q.q0 + row / G) * Hq + g * G + row % G) * (int64_t)D + c * 8);
        *reinterpret_cast<uint4*>(sQ + swz<D>(n, c)) = v;
      }
      if (tid < kRows) {
        const int64_t row = row0 + tid;
        sL[tid] = row < row_end ? a.lse[(q.q0 + row / G) * Hq + g * G + row % G] * kLog2e : 0.f;
      }
      __syncthreads();
      float acc[kRows / 8][4] = {};
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t af[4];
        ldsm_x4(smem_u32(sK) + swz<D>(warp * 16 + (lane & 7) + 8 * ((lane >> 3) & 1), kk * 2 + (lane >> 4)), af);
#pragma unroll
        for (int nt = 0; nt < kRows / 8; nt += 2) {
          uint32_t bf[4];
          ldsm_x4(smem_u32(sQ) + swz<D>(nt * 8 + (lane & 7) + 8 * (lane >> 4), kk * 2 + ((lane >> 3) & 1)), bf);
          mma_bf16(acc[nt], af, bf[0], bf[1]);
          mma_bf16(acc[nt + 1], af, bf[2], bf[3]);
        }
      }
      float part[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < kRows / 8; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = nt * 8 + 2 * tig + (e & 1);
          const int64_t row = row0 + col;
          const int32_t p = q.sp + (int32_t)(row / G);
          const int32_t j = k0 + warp * 16 + gid + 8 * (e >> 1);
          const bool vis = row < row_end && j <= p && (W < 0 || p - j <= W || j < a.num_sink);
          if (vis) part[e >> 1] += ex2(acc[nt][e] * a.sm_scale_log2 - sL[col]);
        }
      }
      sum[0] += part[0];
      sum[1] += part[1];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = sum[e];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      const int k = warp * 16 + gid + 8 * e;
      if (tig == 0 && k < nk && mass_seen(a, q, rel0 + k)) {
        const int32_t page = mass_page(a.plan, q, rel0 + k, ps, a.pool.num_pages);
        if (page < a.pool.num_pages) mass_store(a, q, page, g, rel0 + k, s);
        else atomicOr(a.status, kStatusBounds);
      }
    }
  }
}

template <int D>
cudaError_t launch_mass_mma(const MassArgs& m, int32_t max_keys, cudaStream_t stream) {
  constexpr int smem = (kKeys + kRows) * D * 2 + kRows * 4;
  static PerDeviceOnce setup;
  int dev = 0, unused = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = setup.get(dev, [](int*) {
    return cudaFuncSetAttribute(mass_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  }, &unused);
  if (e != cudaSuccess) return e;
  const int32_t tiles = (max_keys + kKeys - 1) / kKeys;
  const int64_t grid = (int64_t)tiles * m.attn.pool.num_kv_heads * m.attn.plan.num_req;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  mass_prefill_kernel<D><<<(unsigned)grid, kMassThreads, smem, stream>>>(m, tiles);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mass_decode(const MassArgs& m, cudaStream_t stream) {
  const int32_t blocks = (m.attn.max_keys + kDecThreads - 1) / kDecThreads;
  const int64_t grid = (int64_t)blocks * m.attn.plan.num_req;
  if (grid == 0) return cudaSuccess;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  mass_decode_kernel<<<(unsigned)grid, kDecThreads, m.attn.num_qo_heads * sizeof(float), stream>>>(m, blocks);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_mass_prefill(const MassArgs& m, int32_t head_dim, cudaStream_t stream) {
  if (m.attn.max_keys <= 0 || m.attn.plan.num_req == 0) return cudaSuccess;
  if (attn_tc_supported(head_dim, m.attn.group, m.attn.pool.page_size))
    return launch_mass_prefill_tc(m, head_dim, stream);
  return head_dim == 256 ? launch_mass_mma<256>(m, m.attn.max_keys, stream)
                         : launch_mass_mma<512>(m, m.attn.max_keys, stream);
}

}  // namespace pg
