// Key walk of bounded-cache attention: a sliding window plus the first num_sink positions.
//
// Key j is visible from query position p iff
//   kv_start <= j < kv_len,  j <= p,  and  (W < 0  or  p - j <= W  or  j < num_sink).
// A kernel walks the keys in tiles aligned from the first key held. The tiles some row of a
// query tile sees are the sink tiles [0, ns) and the window tiles [ft, ft + wt); where the two
// meet or overlap they are walked as one run, so no key is visited twice.
#pragma once

#include <stdint.h>

namespace pg {

// The low n of 64 bits.
__device__ __forceinline__ uint64_t bits_below(int32_t n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

struct KeyWalk {
  int32_t ns, ft, total;  // sink tiles, first window tile, tiles in all
  int32_t lo, hi;         // the window part's keys [lo, hi); sinks lie below min(num_sink, hi)
  // tile number (from the first key held) of the i-th tile walked
  __device__ __forceinline__ int32_t tile(int32_t i) const { return i < ns ? i : ft + (i - ns); }
};

__device__ __forceinline__ KeyWalk key_walk(int32_t W, int32_t num_sink, int32_t kv_start,
                                            int32_t kv_len, int32_t p_first, int32_t p_last,
                                            int32_t tile) {
  KeyWalk k;
  k.hi = min(p_last + 1, kv_len);
  k.lo = W >= 0 ? max(kv_start, p_first - W) : kv_start;
  k.ns = k.ft = k.total = 0;
  if (k.hi <= kv_start) return k;
  const int32_t se = W >= 0 ? min(num_sink, k.hi) : kv_start;
  k.ns = se > kv_start ? (se - kv_start + tile - 1) / tile : 0;
  if (k.hi <= k.lo) {  // the keys end before the window begins: sinks only
    k.total = k.ns;
    return k;
  }
  k.ft = (k.lo - kv_start) / tile;
  if (k.ns >= k.ft) k.ns = k.ft = 0;  // one run from the first key
  k.total = k.ns + (k.hi - 1 - kv_start) / tile - k.ft + 1;
  return k;
}

}  // namespace pg
