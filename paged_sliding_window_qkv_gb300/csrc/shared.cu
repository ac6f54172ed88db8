// Attention over a shared prefix: the join of a row's parts.
//
// The requests of a group see the same prefix keys, so their query rows (tokens x the heads of a KV
// head) are one block of MMA rows against the prefix: its K and V tiles are read once for all of
// them, and the product is a matrix product where decode has a few rows a request. Where a batch has
// fewer row tiles than the GPU has clusters, the prefix is cut along its keys (attn_tc.cu, PART):
// part i of row t leaves its mean o_i, reference m_i and sum l_i (of weights 2^(s - m_i)). With
// the row's own keys (bf16 mean o, lse) the whole is
//   M = max(m_i, lse / ln 2),  w_i = l_i 2^(m_i - M),  w = 2^(lse / ln 2 - M)
//   out = (sum w_i o_i + w o) / (sum w_i + w),  lse' = (M + log2(sum w_i + w)) ln 2
// A block takes one row, four columns a thread, eight parts in flight.
#include "pg_internal.h"

#include <cuda_bf16.h>
#include <math.h>

namespace pg {
namespace {

constexpr int kParts = 8;

template <int D>
__global__ void __launch_bounds__(D / 4) shared_join_kernel(SharedJoinArgs a) {
  const int64_t rows = (int64_t)a.num_tokens * a.num_qo_heads, row = blockIdx.x;
  const int32_t n = a.tok_parts[row / a.num_qo_heads];
  if (n == 0) return;
  const int c = threadIdx.x;
  uint2* const dst = reinterpret_cast<uint2*>(a.out + row * D) + c;
  const uint2 own = *dst;
  const float own_lse = a.lse[row];
  float M = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m, float l, float4 x) {
    if (l == 0.f) return;  // saw no key (a NaN sum stays)
    const float mn = fmaxf(M, m), so = exp2f(M - mn), w = l * exp2f(m - mn);
    acc.x = acc.x * so + w * x.x;
    acc.y = acc.y * so + w * x.y;
    acc.z = acc.z * so + w * x.z;
    acc.w = acc.w * so + w * x.w;
    den = den * so + w;
    M = mn;
  };
  for (int32_t i0 = 0; i0 < n; i0 += kParts) {
    float2 ml[kParts];
    float4 v[kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const bool in = i0 + k < n;
      const int64_t at = (i0 + k) * rows + row;
      ml[k] = in ? *reinterpret_cast<const float2*>(a.part_ml + 2 * at) : make_float2(-INFINITY, 0.f);
      v[k] = in ? __ldcs(reinterpret_cast<const float4*>(a.part_o + at * D) + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) add(ml[k].x, ml[k].y, v[k]);
  }
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  add(own_lse * 1.4426950408889634f, own_lse == -INFINITY ? 0.f : 1.f,
      make_float4(lo(own.x), hi(own.x), lo(own.y), hi(own.y)));
  const float inv = den != 0.f ? 1.f / den : 0.f;
  auto pack = [](float x, float y) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
  };
  __syncthreads();  // every thread has read the row's lse
  *dst = make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
  if (c == 0) a.lse[row] = den != 0.f ? (M + log2f(den)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_shared_join(const SharedJoinArgs& a, int32_t head_dim, cudaStream_t stream) {
  const unsigned grid = (unsigned)((int64_t)a.num_tokens * a.num_qo_heads);
  if (head_dim == 256) shared_join_kernel<256><<<grid, 64, 0, stream>>>(a);
  else shared_join_kernel<512><<<grid, 128, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace pg
