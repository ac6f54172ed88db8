// Read-back of an 8-bit pool: code * 2^e of every key that a plan's requests hold, into the same
// pages of a bf16 pool, or, for an attention call on the bf16 kernels, the pages that the call reads
// into a workspace in the order of the plan's page list.
//
// HBM-bound: 1 byte in and 2 out an element, and nothing to compute but the conversion (exact). A
// warp takes one (layer, page of the list, K or V, head) in pieces of 256 codes, 8 a lane, so that a
// store instruction writes 512 contiguous bytes, with sixteen loads in flight. 32 requests of up to 16384 keys,
// two layers, head_dim 512: 259 us, 6.7 TB/s; one of 4097 keys 4.4 us (7 before it started while the
// stream's previous kernel ends).
#include "pg_internal.h"
#include "q8.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace pg {
namespace {

constexpr int kWarps = 8;

// The request that holds entry i of the page list: the last r with indptr[r] <= i.
__device__ __forceinline__ int32_t request_of(const PlanDev& pl, int32_t i, int lane) {
  int32_t lo = 0, n = pl.num_req;  // in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) / 32, at = lo + lane * step;
    const bool in = lane * step < n && pl.kv_page_indptr[at] <= i;
    const int32_t c = __popc(__ballot_sync(0xffffffffu, in)) - 1;  // (entry lo itself always is)
    const int32_t from = lo + max(c, 0) * step;
    n = min(step, lo + n - from);
    lo = from;
  }
  return lo;
}

__device__ __forceinline__ uint32_t bf2(float2 v, float s) {
  __nv_bfloat162 h = __floats2bfloat162_rn(v.x * s, v.y * s);
  return *reinterpret_cast<uint32_t*>(&h);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) dequant_kernel(DequantArgs a) {
  const int lane = threadIdx.x & 31;
  const int32_t heads = 2 * a.num_kv_heads, ps = a.page_size, NP = a.plan.num_page_ids;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (task >= (int64_t)a.num_layers * NP * heads) return;
  const int32_t kvh = (int32_t)(task % heads);
  const int32_t i = (int32_t)(task / heads % NP), layer = (int32_t)(task / heads / NP);
  const PlanDev& pl = a.plan;
  // (launched programmatically: the plan, which copies alone write, is looked at while the stream's
  // previous kernel ends; every warp then waits for that kernel, whatever it has to do)
  bool skip = i >= (a.whole ? *a.whole : pl.kv_page_indptr[pl.num_req]);  // room behind the list
  const int32_t page = skip ? -1 : pl.page_at(i);
  int32_t rows = ps;  // slots of the page that hold keys
  bool seen = true;
  if (!skip && !a.whole) {
    const int32_t r = request_of(pl, i, lane);
    if (i + 1 == pl.kv_page_indptr[r + 1]) rows = min(ps, pl.last_page_len[r]);
    if (a.list && a.window_left >= 0) {
      // a page that lies between the sinks and the first query's window is not read
      const int64_t first = (int64_t)pl.kv_start[r] + (int64_t)(i - pl.kv_page_indptr[r]) * ps;
      const int64_t lo = (int64_t)pl.start_pos[r] - a.window_left;
      seen = first + ps > lo || first < a.num_sink;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (skip) return;
  if (!seen) return;
  const bool good = page >= 0 && page < a.num_pages;
  if (!good) {
    if (lane == 0) atomicOr(a.status, kStatusBounds);
    if (!a.list) return;
  }
  const int64_t src_row = layer * a.src.rows_layer + ((int64_t)page * heads + kvh) * ps;
  const uint8_t* const codes = a.src.codes + src_row * D;
  const uint8_t* const scales = a.src.scales + src_row;
  __nv_bfloat16* const dst =
      a.dst + layer * a.dst_stride_layer + ((int64_t)(a.list ? i : page) * heads + kvh) * ps * D;
  constexpr int kBatch = 16, PIECES = D / 256;  // a piece: 256 codes of a row
  const int32_t pieces = rows * PIECES;
  for (int32_t p0 = 0; p0 < pieces; p0 += kBatch) {
    uint2 c[kBatch];
    uint32_t s[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t p = p0 + k;
      const bool in = good && p < pieces;
      c[k] = in ? __ldcs(reinterpret_cast<const uint2*>(codes + (int64_t)p * 256) + lane) : make_uint2(0u, 0u);
      s[k] = in ? scales[p / PIECES] : 127u;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t p = p0 + k;
      if (p >= pieces) break;
      const float f = q8_scale(s[k]);
      *(reinterpret_cast<uint4*>(dst + (int64_t)p * 256) + lane) =
          make_uint4(bf2(q8_values(c[k].x & 0xFFFFu), f), bf2(q8_values(c[k].x >> 16), f),
                     bf2(q8_values(c[k].y & 0xFFFFu), f), bf2(q8_values(c[k].y >> 16), f));
    }
  }
}

}  // namespace

cudaError_t launch_dequant(const DequantArgs& a, cudaStream_t stream) {
  const int64_t tasks = (int64_t)a.num_layers * a.plan.num_page_ids * 2 * a.num_kv_heads;
  if (tasks == 0) return cudaSuccess;
  const unsigned grid = (unsigned)((tasks + kWarps - 1) / kWarps);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.head_dim == 256 ? cudaLaunchKernelEx(&cfg, dequant_kernel<256>, a)
                                          : cudaLaunchKernelEx(&cfg, dequant_kernel<512>, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace pg
