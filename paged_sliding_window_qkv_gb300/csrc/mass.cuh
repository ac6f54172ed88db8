// What the kernels that accumulate attention weights share: a request's geometry, the page of a
// key, the query tiles that see a tile of keys, and the update of a key's statistics.
#pragma once

#include "pg_internal.h"

namespace pg {

struct MassReq {
  int32_t q0, len, sp, kvp0, kvp1, ks0, n;  // n: keys held, positions [ks0, ks0 + n)
};
__device__ __forceinline__ MassReq mass_req(const PlanDev& pl, int32_t r, int32_t ps) {
  MassReq q;
  q.q0 = pl.qo_indptr[r];
  q.len = pl.qo_indptr[r + 1] - q.q0;
  q.sp = pl.start_pos[r];
  q.kvp0 = pl.kv_page_indptr[r];
  q.kvp1 = pl.kv_page_indptr[r + 1];
  q.ks0 = pl.kv_start[r];
  q.n = (q.kvp1 - q.kvp0 - 1) * ps + pl.last_page_len[r];
  return q;
}

// Page holding key index rel of the request (num_pages when the metadata is out of range).
__device__ __forceinline__ int32_t mass_page(const PlanDev& pl, const MassReq& q, int32_t rel,
                                             int32_t ps, int32_t num_pages) {
  const int32_t pidx = q.kvp0 + rel / ps;
  const int32_t p = (pidx < q.kvp1 && pidx < pl.num_page_ids) ? pl.page_ids[pidx] : num_pages;
  return p < 0 || p >= num_pages ? num_pages : p;
}

// Query tiles [first, end) of 256 rows (256 / group tokens, from the request's first token) in
// which some row sees some key of the kt-th 256 keys.
struct MassTiles {
  int32_t first, end;
};
__device__ __forceinline__ MassTiles mass_tiles(const AttnArgs& a, const MassReq& q, int32_t kt) {
  MassTiles t{0, 0};
  const int32_t rel0 = kt * 256;
  if (rel0 >= q.n) return t;
  const int32_t k0 = q.ks0 + rel0, k1 = q.ks0 + min(q.n, rel0 + 256) - 1;
  const int32_t tq = 256 / a.group;
  const int32_t tok0 = max(0, k0 - q.sp);
  int64_t tok1 = q.len;
  if (a.window_left >= 0 && k0 >= a.num_sink)
    tok1 = min(tok1, (int64_t)k1 + a.window_left - q.sp + 1);
  if (tok0 >= tok1) return t;
  t.first = tok0 / tq;
  t.end = (int32_t)((tok1 - 1) / tq) + 1;
  return t;
}

// Whether some row of the step sees key index rel: the first position at or past the key's is the
// one that sees most of what lies before it. (The statistics of a key that no row sees stay
// as they are, bit for bit: +0 would make +0 of -0.)
__device__ __forceinline__ bool mass_seen(const AttnArgs& a, const MassReq& q, int32_t rel) {
  const int32_t j = q.ks0 + rel;
  return j < q.sp + q.len && (a.window_left < 0 || j < a.num_sink || max(j, q.sp) - j <= a.window_left);
}

// mass and position of one key: keys that the step wrote are set, older ones add
__device__ __forceinline__ void mass_store(const AttnArgs& a, const MassReq& q, int32_t page,
                                           int32_t g, int32_t rel, float sum) {
  const int32_t ps = a.pool.page_size, j = q.ks0 + rel;
  const int64_t at = ((int64_t)page * a.pool.num_kv_heads + g) * ps + rel % ps;
  if (j >= q.sp) {
    a.stats.mass[at] = sum;
    a.stats.pos[at] = j;
  } else {
    a.stats.mass[at] += sum;
  }
}

}  // namespace pg
