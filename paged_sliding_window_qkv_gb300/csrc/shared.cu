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
// (Of a decode step it is the join of the own keys' records that takes the parts along, in
// attn_bounded_decode.cu; this kernel is for steps of more tokens.) Bound by the records' bytes: a row a warp, everything
// on its way before it is added, 23 us of 8 prompts behind 4096 keys at head_dim 512 (76 with a block of columns).
#include "pg_internal.h"

#include <cuda_bf16.h>
#include <math.h>

namespace pg {
namespace {

constexpr int kJoinWarps = 8;

// A warp takes a row: D / 32 columns a lane as quads 32 lanes apart, everything it reads on its way
// before anything is added up.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_kernel(SharedJoinArgs a) {
  constexpr int Q = D / 128;  // quads a lane
  const int64_t rows = (int64_t)a.num_tokens * a.num_qo_heads;
  const int64_t row = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  const int32_t n = a.tok_parts[row / a.num_qo_heads];
  const float own_lse = a.own_lse[row];
  if (n == 0) {
    if (a.lse && lane == 0) a.lse[row] = own_lse;
    return;
  }
  uint2* const dst = reinterpret_cast<uint2*>(a.out + row * D) + lane;
  uint2 own[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) own[q] = dst[32 * q];
  float M = -INFINITY, den = 0.f;
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  // weight of a state (m, l), everything before it moved to the new reference
  auto weigh = [&](float m, float l) {
    const float mn = fmaxf(M, m), so = exp2f(M - mn), w = l * exp2f(m - mn);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      acc[q].x *= so; acc[q].y *= so; acc[q].z *= so; acc[q].w *= so;
    }
    den = den * so + w;
    M = mn;
    return w;
  };
  auto add = [&](int q, float w, float4 x) {
    acc[q].x += w * x.x; acc[q].y += w * x.y; acc[q].z += w * x.z; acc[q].w += w * x.w;
  };
  for (int32_t i = 0; i < n; ++i) {
    const int64_t at = i * rows + row;
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
    float4 v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = __ldcs(reinterpret_cast<const float4*>(a.part_o + at * D) + lane + 32 * q);
    if (ml.y == 0.f) continue;  // saw no key (a NaN sum stays)
    const float w = weigh(ml.x, ml.y);
#pragma unroll
    for (int q = 0; q < Q; ++q) add(q, w, v[q]);
  }
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  if (own_lse != -INFINITY) {
    const float w = weigh(own_lse * 1.4426950408889634f, 1.f);
#pragma unroll
    for (int q = 0; q < Q; ++q) add(q, w, make_float4(lo(own[q].x), hi(own[q].x), lo(own[q].y), hi(own[q].y)));
  }
  const float inv = den != 0.f ? 1.f / den : 0.f;
  auto pack = [](float x, float y) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
  };
#pragma unroll
  for (int q = 0; q < Q; ++q)
    dst[32 * q] = make_uint2(pack(acc[q].x * inv, acc[q].y * inv), pack(acc[q].z * inv, acc[q].w * inv));
  if (a.lse && lane == 0) a.lse[row] = den != 0.f ? (M + log2f(den)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_shared_join(const SharedJoinArgs& a, int32_t head_dim, cudaStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)a.num_tokens * a.num_qo_heads + kJoinWarps - 1) / kJoinWarps);
  if (head_dim == 256) shared_join_kernel<256><<<grid, kJoinWarps * 32, 0, stream>>>(a);
  else shared_join_kernel<512><<<grid, kJoinWarps * 32, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace pg
