// Host side of the C ABI: plan builder, checked geometry, argument checks, dispatch.
//
// Every check runs before any launch and before any write to caller memory
// ("feat(kernels): Rust wrapper for the hd256 windowed paged prefill", Description and
// Verification; "gemma4: serving prep needs pool-write forms", Proposed Plan).
#include "../../include/pg.h"
#include "pg_internal.h"

#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <memory>
#include <exception>
#include <mutex>
#include <new>
#include <algorithm>
#include <vector>

namespace pg {

static std::atomic<int64_t> g_launches{0};
void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

// Bounded waits give up after two seconds unless the test hook set a shorter limit.
constexpr uint64_t kDefaultWaitNs = 2000000000ull;
static std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};
static std::atomic<int32_t> g_test_withhold{0};
void wait_settings(uint64_t* wait_ns, int32_t* test_withhold) {
  *wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  *test_withhold = g_test_withhold.load(std::memory_order_relaxed);
}

// One status word per device, allocated on first use with that device current.
static std::mutex g_status_mu;
static int* g_status_dev[128] = {nullptr};

static int* status_word(int* err) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) {
    *err = PG_ERR_CUDA;
    return nullptr;
  }
  std::lock_guard<std::mutex> lk(g_status_mu);
  if (!g_status_dev[dev]) {
    int* p = nullptr;
    if (cudaMalloc(&p, sizeof(int)) != cudaSuccess) { *err = PG_ERR_CUDA; return nullptr; }
    if (cudaMemset(p, 0, sizeof(int)) != cudaSuccess) { cudaFree(p); *err = PG_ERR_CUDA; return nullptr; }
    g_status_dev[dev] = p;
  }
  *err = PG_OK;
  return g_status_dev[dev];
}

// ------------------------------------------------------------------ checked arithmetic
static bool mul_i64(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
static bool add_i64(int64_t a, int64_t b, int64_t* out) { return !__builtin_add_overflow(a, b, out); }
static bool fits_i32(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }

// Query tokens per prefill CTA as the plan derives it (must agree with the kernel's):
// 128 rows on the tensor-memory path (head_dim 256/512, group dividing 128, power-of-two page
// size >= 8), else 64 (head_dim 256) or 32 (head_dim 512) rows on the mma.sync path.
static int32_t plan_cta_tile_q(int32_t head_dim, int32_t group, int32_t page_size) {
  if (group <= 0 || group > 16) return 0;
  const bool tc = (head_dim == 256 || head_dim == 512) && 128 % group == 0 && page_size >= 8 &&
                  (page_size & (page_size - 1)) == 0;
  const int32_t rows = tc ? 128 : head_dim == 256 ? 64 : head_dim == 512 ? 32 : 0;
  if (rows == 0 || rows % group != 0) return 0;
  return rows / group;
}
static int32_t plan_kv_chunk(int32_t head_dim) { return head_dim == 512 ? 512 : 256; }

}  // namespace pg

using namespace pg;

// Pinned host staging for a plan's metadata upload, two buffers used alternately: an upload from
// pageable memory can hold the host until the stream reaches it, which in a serving loop that
// rebuilds a plan while earlier calls still run would stall every later launch. Buffer k is
// rewritten only after the upload recorded on done[k] (two builds back) has completed.
struct PlanStage {
  int32_t* host[2] = {nullptr, nullptr};
  size_t cap[2] = {0, 0};
  cudaEvent_t done[2] = {nullptr, nullptr};
  int next = 0;
};

// The parts that a plan's prefixes are cut into.
struct PartSet {
  int32_t num = 0;
  int32_t beside = 0;  // decode: SMs that the parts leave to the own keys (0: one after the other)
  bool plain = true;   // every request reads its prefix itself: by the estimate that is sooner
  size_t o_tab = 0, o_row = 0, o_live = 0, o_tok = 0;  // pair table, record rows, counts, parts of each token
};

struct pg_plan {
  int32_t num_req = 0, num_tokens = 0, num_qo_heads = 0, num_kv_heads = 0, head_dim = 0,
          page_size = 0;
  int32_t max_page_id = -1, max_last_page_len = 0, max_qo_len = 0, max_kv_len = 0,
          max_pos_end = 0;
  int32_t cta_tile_q = 0, decode = 0, kv_chunk = 0, max_chunks = 0, num_work = 0, num_pairs = 0;
  int32_t num_page_ids = 0;
  int32_t ring = 0, ring_window = -1;  // ring addressing (window-crossing requests) and its window
  // key segments (cascade attention): request r's pages hold key positions
  // [kv_start_r, kv_start_r + n_r); prep_ok: every request's step tokens are its segment's tail
  int32_t segment = 0, prep_ok = 1;
  cudaStream_t stream = nullptr;
  int device = 0;
  int32_t* dev = nullptr;  // one device allocation holding every metadata array
  size_t dev_elems = 0;
  size_t dev_cap = 0;      // bytes allocated at dev
  // offsets (elements) of each array inside `dev`
  size_t o_qo = 0, o_kvp = 0, o_pages = 0, o_last = 0, o_start = 0, o_kvs = 0, o_tokreq = 0,
         o_wreq = 0, o_wtok = 0, o_pair = 0, o_live = 0;
  int32_t room_work = 0, room_pairs = 0;  // entries that the work and the pair table have room for
  PlanStage stage;  // carried over from build to build of the same plan
  int32_t max_seen = 0;           // the most keys a request holds
  int32_t page_keys = 0;          // the most keys one could hold in as many pages, the others keeping one each
  int64_t tiles = 0;              // tiles of 128 keys over all requests (one KV head)
  std::vector<int32_t> host_ids;  // the page list, for the check below
  mutable int8_t shared = -1;     // a page is listed twice (-1: not looked at yet)
  // shared prefixes (pg_plan_paged_shared; null otherwise): the requests' own keys as a segment plan
  // over arrays in `dev` (it owns nothing there), and the prefixes' parts
  std::unique_ptr<pg_plan> own;
  int32_t num_groups = 0, room_parts = 0, parts_most = 0, prefix_pages = 0;
  size_t o_pre_pages = 0;
  PartSet parts[2];  // over a bf16 pool, and over an 8-bit one
};

namespace {

// releases a plan's staging buffers once their uploads have completed
void free_stage(PlanStage* st) {
  for (int k = 0; k < 2; ++k) {
    if (st->done[k]) {
      cudaEventSynchronize(st->done[k]);
      cudaEventDestroy(st->done[k]);
      st->done[k] = nullptr;
    }
    if (st->host[k]) cudaFreeHost(st->host[k]);
    st->host[k] = nullptr;
    st->cap[k] = 0;
  }
}

// What the kernels of a shared plan take, in us by head_dim (256, 512) and set (bf16, 8-bit pools), as
// measured: decode steps of 1..64 requests, prefixes of 128..8192 keys, 16 and 8 query heads, pages of 8..64
// slots. (Over 192 of them on either kind of pool the form chosen by these took 1.007 times the better form's
// time in the mean on bf16 pools and 1.003 on 8-bit ones, 1.19 at most; the parts alone 1.28 and 1.58.)
struct SharedCost {
  double start[2] = {9, 11};                          // of the parts' kernel
  double tile[2] = {0.7, 1.05}, ends[2] = {4.8, 3.5};  // of its units: 64 keys, start and epilogue
  double dec_start[2][2] = {{9, 11.5}, {10.5, 13.5}};  // of a decode kernel with its join
  double dec_l2[2][2] = {{1.15, 2.8}, {0.6, 2.45}};    // of its tiles of 128 keys: another request's too,
  double dec_dram[2][2] = {{2.5, 5.4}, {1.2, 3.2}};    // or a request's alone
};
constexpr SharedCost kCost;
constexpr double kJoin = 4, kBytesPerUs = 6.5e6;
constexpr double kReadBack = 2, kBackBatch = 1.5;  // a read-back's launch, and each batch of a warp's loads
std::atomic<int32_t> g_test_shared{0};  // test hook: 1 parts, 2 plain, whatever the estimate says

// Groups of consecutive requests that share their first keys.
struct Groups {
  int32_t num = 0;
  const int64_t* indptr = nullptr;
  const int64_t* prefix = nullptr;
};

// SMs of the current device.
int sm_count() {
  static PerDeviceOnce once;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (once.get(dev, [dev](int* v) { return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev); }, &n) !=
      cudaSuccess)
    return 0;
  return n;
}

// One entry of the pair table for every two query tiles of a run of rows (a request, or a group's
// rows before its prefix): see PlanDev.
void put_pairs(std::vector<int32_t>* tab, int32_t tile, int32_t q0, int32_t len, int32_t start, int32_t kvp0,
               int32_t kvp1, int32_t kv_end, int32_t kv_start) {
  for (int64_t t = 0; t < len; t += 2 * (int64_t)tile) {
    const int32_t e[8] = {(int32_t)t, q0, len, start, kvp0, kvp1, kv_end, kv_start};
    tab->insert(tab->end(), e, e + 8);
  }
}
// The pairs that see the most keys come first (a window keeps that order): on 8 prompts of
// 384..2026 tokens the busiest cluster then has 4% more than the mean, against 22% request by
// request.
void sort_pairs(std::vector<int32_t>* tab, int32_t tile, bool sort) {
  const size_t n = tab->size() / 8;
  std::vector<int32_t> order(n), sorted(tab->size());
  for (size_t i = 0; i < n; ++i) order[i] = (int32_t)i;
  auto seen = [&](int32_t i) {
    const int32_t* e = tab->data() + 8 * (size_t)i;
    const int64_t end = (int64_t)e[3] + std::min<int64_t>((int64_t)e[0] + 2 * (int64_t)tile, e[2]);
    return std::min<int64_t>(end, e[6]) - e[7];
  };
  if (sort) std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) { return seen(x) < seen(y); });
  std::reverse(order.begin(), order.end());
  for (size_t i = 0; i < n; ++i) std::copy_n(tab->data() + 8 * (size_t)order[i], 8, sorted.data() + 8 * i);
  tab->swap(sorted);
}

// The most parts that a prefix is cut into, for as many tokens and groups whatever their lengths (the
// records' room, which captured calls keep): enough for one unit a cluster, and four where there are
// fewer than two rounds of units anyway.
int32_t most_parts(int32_t tokens, int32_t groups, int32_t tile, int32_t units_per_pair, int32_t sms) {
  const int64_t pairs = std::max<int64_t>(groups, ((int64_t)tokens + 2 * tile - 1) / (2 * tile));
  const int64_t units = std::max<int64_t>(1, pairs * units_per_pair), clusters = std::max(1, sms / 2);
  if (2 * units <= clusters) return (int32_t)std::min<int64_t>(clusters / units, 64);
  return units <= 2 * clusters ? 4 : 1;
}

// ring_window < 0: linear addressing (slot = position, pages cover [0, kv_len) exactly, with
// last_page_len). ring_window >= 0: ring addressing for window-crossing requests: logical page
// pos / ps lives in the request's page (pos / ps) mod (pages held), kv_len = start_pos + qo_len,
// last_page_len is not read, and the ring must hold the window plus the step
// (pages * ps >= ring_window + qo_len), so no key a query of the step can see is overwritten by
// the step's own writes.
// kv_start != null: key segments (linear addressing within the segment): request r's pages hold
// key positions [kv_start_r, kv_start_r + n_r), n_r = (pages - 1) * ps + last_page_len_r, from
// slot 0 on; the segment ends at or before the step's last position.
int build_plan(pg_plan* p, int32_t num_req, const int64_t* qo_indptr,
               const int64_t* kv_page_indptr, const int32_t* page_ids,
               const int32_t* last_page_len, const int64_t* start_pos, int32_t Hq,
               int32_t Hkv, int32_t D, int32_t ps, cudaStream_t stream,
               int32_t ring_window = -1, const int64_t* kv_start = nullptr, const Groups* groups = nullptr) {
  const bool ring = ring_window >= 0;
  const bool segment = kv_start != nullptr;
  if (ring && segment) return PG_ERR_ARG;
  // The head relation is settled before anything divides by num_kv_heads.
  if (Hkv == 0) return PG_ERR_ZERO_KV_HEADS;
  if (Hkv < 0 || Hq <= 0 || Hq % Hkv != 0) return PG_ERR_HEADS;
  if (D <= 0 || D % 2 != 0 || ps <= 0) return PG_ERR_ARG;
  if (num_req < 0) return PG_ERR_ARG;
  if (num_req > 0 && (!qo_indptr || !kv_page_indptr || !page_ids || !start_pos ||
                      (!ring && !last_page_len)))
    return PG_ERR_ARG;
  const int32_t group = Hq / Hkv;

  std::vector<int32_t> qo((size_t)num_req + 1, 0), kvp((size_t)num_req + 1, 0), last(num_req), start(num_req),
      kvs(num_req, 0);
  if (num_req > 0) {
    if (qo_indptr[0] != 0 || kv_page_indptr[0] != 0) return PG_ERR_ARG;
  }
  int32_t max_page = -1, max_last = 0, max_qo = 0, max_kv = 0, max_end = 0, max_seen = 0;
  int64_t tiles = 0;
  bool all_one = num_req > 0, prep_ok = true;
  for (int32_t r = 0; r < num_req; ++r) {
    const int64_t q0 = qo_indptr[r], q1 = qo_indptr[r + 1];
    const int64_t k0 = kv_page_indptr[r], k1 = kv_page_indptr[r + 1];
    if (q1 <= q0 || k1 <= k0) return PG_ERR_ARG;  // every request: >= 1 token, >= 1 page
    if (!fits_i32(q1) || !fits_i32(k1)) return PG_ERR_I32_OVERFLOW;
    const int64_t qo_len = q1 - q0;
    const int64_t sp = start_pos[r];
    if (sp < 0) return PG_ERR_ARG;
    int64_t pos_end = 0;
    if (!add_i64(sp, qo_len, &pos_end) || !fits_i32(pos_end)) return PG_ERR_I32_OVERFLOW;
    int32_t lpl = 0;
    int64_t kv_len = 0, seg0 = 0;  // kv_len: end of the keys held (exclusive); seg0: first
    if (!ring) {
      lpl = last_page_len[r];
      if (lpl < 1 || lpl > ps) return PG_ERR_LAST_PAGE_LEN;
      if (!mul_i64(k1 - k0 - 1, ps, &kv_len) || !add_i64(kv_len, lpl, &kv_len))
        return PG_ERR_I32_OVERFLOW;
      if (segment) {
        seg0 = kv_start[r];
        if (seg0 < 0) return PG_ERR_ARG;
        if (!add_i64(seg0, kv_len, &kv_len)) return PG_ERR_I32_OVERFLOW;
      }
      if (!fits_i32(kv_len)) return PG_ERR_I32_OVERFLOW;
      if (!segment && kv_len != pos_end) return PG_ERR_COVERAGE;
      // a segment holds no key past the step's last position (no query could see it)
      if (segment && kv_len > pos_end) return PG_ERR_COVERAGE;
      if (segment && !(kv_len == pos_end && sp >= seg0)) prep_ok = false;
    } else {
      int64_t cap = 0, need = 0;
      if (!mul_i64(k1 - k0, ps, &cap) || !add_i64(ring_window, qo_len, &need))
        return PG_ERR_I32_OVERFLOW;
      // a step's write can cover a key one of its queries sees only if some position wraps
      // (pos_end > cap) and the ring is shorter than the window plus the step
      if (cap < need && pos_end > cap) return PG_ERR_COVERAGE;
      kv_len = pos_end;
      // the position's slot in its (ring) page; last_page_len is not used in ring addressing
      lpl = (int32_t)(pos_end - ((pos_end - 1) / ps) * ps);
    }
    qo[r + 1] = (int32_t)q1;
    kvp[r + 1] = (int32_t)k1;
    last[r] = lpl;
    start[r] = (int32_t)sp;
    kvs[r] = (int32_t)seg0;
    if (kv_len - seg0 > max_seen) max_seen = (int32_t)(kv_len - seg0);
    tiles += (kv_len - seg0 + 127) / 128;
    if (lpl > max_last) max_last = lpl;
    if (qo_len > max_qo) max_qo = (int32_t)qo_len;
    if (kv_len > max_kv) max_kv = (int32_t)kv_len;
    if (pos_end > max_end) max_end = (int32_t)pos_end;
    if (qo_len != 1) all_one = false;
  }
  const int32_t T = num_req > 0 ? qo[num_req] : 0;
  const int32_t NP = num_req > 0 ? kvp[num_req] : 0;
  for (int32_t i = 0; i < NP; ++i) {
    if (page_ids[i] < 0) return PG_ERR_PAGE_OOB;
    if (page_ids[i] > max_page) max_page = page_ids[i];
  }

  // Tiling derived from the geometry; attention re-derives it from the kernel itself.
  const int32_t cta = plan_cta_tile_q(D, group, ps);
  const int32_t chunk = plan_kv_chunk(D);
  {
    // the chunked decode kernel holds a request's key chunks in its grid's z dimension
    const int64_t seen = ring ? std::min<int64_t>(max_kv, (int64_t)ring_window + 1) : max_seen;
    if (all_one && !attn_decode_stream_supported(D, group, ps) && (seen + chunk - 1) / chunk > 65535)
      return PG_ERR_I32_OVERFLOW;
  }
  int64_t nwork = 0;
  std::vector<int32_t> wreq, wtok, ptab;
  if (cta > 0) {
    for (int32_t r = 0; r < num_req; ++r) {
      const int32_t len = qo[r + 1] - qo[r];
      for (int32_t t = 0; t < len; t += cta) {
        wreq.push_back(r);
        wtok.push_back(t);
      }
      // the tcgen05 prefill runs query tiles in pairs (one per CTA of a cluster) that share
      // their key tiles; a request with an odd number of tiles ends with a single-tile pair
      const int32_t kv_len =
          ring ? start[r] + len : kvs[r] + (kvp[r + 1] - kvp[r] - 1) * ps + last[r];
      put_pairs(&ptab, cta, qo[r], len, start[r], kvp[r], kvp[r + 1], kv_len, kvs[r]);
    }
    nwork = (int64_t)wreq.size();
    if (!all_one) sort_pairs(&ptab, cta, num_req > 1);  // (decode looks requests up in the table)
  }
  if (!fits_i32(nwork)) return PG_ERR_I32_OVERFLOW;
  // A graph that captured the plan's calls holds the addresses of these arrays, so an update to as many
  // requests, tokens and pages has to find each at its place however the tokens are spread: the tables
  // have room for the most tiles that any such plan has (a last one a request, and whole ones).
  const int32_t npairs = (int32_t)(ptab.size() / 8);
  const int32_t room_work = cta > 0 && num_req > 0 ? num_req + (T - num_req) / cta : 0;
  const int32_t room_pairs = cta > 0 && num_req > 0 ? num_req + (T - num_req) / (2 * cta) : 0;
  wreq.resize((size_t)room_work, 0);
  wtok.resize((size_t)room_work, 0);
  ptab.resize((size_t)room_pairs * 8, 0);
  const int32_t live[2] = {(int32_t)nwork, npairs};

  // Shared prefixes: the requests' own keys as segments, and the parts of each group's prefix.
  struct Parts {
    std::vector<int32_t> tab, row, tok;
    int32_t num = 0, beside = 0;
    bool plain = true;
  } parts[2];
  std::vector<int32_t> kvp2, kvs2, pages2, ptab2, pre_pages;
  int32_t seen2 = 0, room_parts = 0, parts_most = 0;
  int64_t tiles2 = 0, tiles_l2 = 0;  // of 128 keys: own ones, and those that an earlier request has read
  if (groups) {
    if (!attn_tc_supported(D, group, ps) || cta <= 0) return PG_ERR_PLAN_MISMATCH;
    if (groups->num < 0 || (groups->num > 0 && (!groups->indptr || !groups->prefix))) return PG_ERR_ARG;
    if ((groups->num == 0) != (num_req == 0)) return PG_ERR_ARG;
    if (groups->num > 0 && (groups->indptr[0] != 0 || groups->indptr[groups->num] != num_req)) return PG_ERR_ARG;
    kvp2.push_back(0);
    std::vector<int32_t> pre(groups->num);
    for (int32_t g = 0; g < groups->num; ++g) {
      const int64_t r0 = groups->indptr[g], r1 = groups->indptr[g + 1], len = groups->prefix[g];
      if (r1 <= r0 || r1 > num_req) return PG_ERR_ARG;
      if (len < 0) return PG_ERR_ARG;
      if (len % ps != 0) return PG_ERR_COVERAGE;
      for (int64_t r = r0; r < r1; ++r) {
        if (len > start[r]) return PG_ERR_COVERAGE;
        const int32_t n = (int32_t)(len / ps);
        if (!std::equal(page_ids + kvp[r], page_ids + kvp[r] + n, page_ids + kvp[r0])) return PG_ERR_COVERAGE;
        pages2.insert(pages2.end(), page_ids + kvp[r] + n, page_ids + kvp[r + 1]);
        kvp2.push_back((int32_t)pages2.size());
        kvs2.push_back((int32_t)len);
        const int32_t held = (kvp[r + 1] - kvp[r] - 1) * ps + last[r] - (int32_t)len;
        seen2 = std::max(seen2, held);
        tiles2 += (held + 127) / 128;
        put_pairs(&ptab2, cta, qo[r], qo[r + 1] - qo[r], start[r], kvp2[r], kvp2[r + 1], held + (int32_t)len,
                  (int32_t)len);
      }
      pre[g] = (int32_t)len;
      tiles_l2 += (r1 - r0 - 1) * (len / 128);
      pre_pages.insert(pre_pages.end(), page_ids + kvp[r0], page_ids + kvp[r0] + len / ps);
    }
    if (!all_one) sort_pairs(&ptab2, cta, num_req > 1);
    const int32_t heads = Hkv * (D / 256), sms = std::max(2, sm_count()), step = std::max(64, ps);
    const int32_t dx = D == 512 ? 1 : 0;
    parts_most = num_req > 0 ? most_parts(T, groups->num, cta, heads, sms) : 0;
    // room for what any batch of as many groups, requests, tokens and pages needs
    room_parts = num_req > 0 ? (groups->num + (T - groups->num) / (2 * cta)) * parts_most : 0;
    const int32_t most_len = pre.empty() ? 0 : *std::max_element(pre.begin(), pre.end());
    auto tokens_of = [&](int32_t g) { return qo[groups->indptr[g + 1]] - qo[groups->indptr[g]]; };
    auto pairs_of = [&](int32_t g) { return ((int64_t)tokens_of(g) + 2 * cta - 1) / (2 * cta); };
    auto steps_of = [&](int32_t g) { return ((int64_t)pre[g] + step - 1) / step; };
    for (int set = 0; set < 2; ++set) {
      Parts& p = parts[set];
      // Over 8-bit pools whose pages the decode on codes does not take, own keys and the plain walk go over a
      // read-back with the bf16 kernel, one after the other; the plain walk's repeats the prefixes.
      const bool back = set == 1 && !q8_decode_supported(D, group, ps);
      const int cs = back ? 0 : set;  // whose kernel
      // (a warp takes a page of a head, in batches of 16 x 256 codes)
      auto back_us = [&](size_t n) {
        return kReadBack + kBackBatch * ((ps * (D / 256) + 15) / 16) + (double)n * 6 * Hkv * ps * D / kBytesPerUs;
      };
      // How long a part is (in steps of 64 keys, or a page; a group is cut into as few of one length):
      // every candidate costs rounds of units over the clusters, each as long as its key tiles, a start and
      // an epilogue. A decode step's own keys run beside the parts, on SMs left free for them, where that
      // ends sooner: a CTA takes about 8 us to begin and end and 6.5 for a tile of 128 keys at head_dim 512,
      // 4 in 8 bits.
      auto own_us = [&](int32_t on) {
        return 8 + (cs == 0 ? 6.5 : 4.0) * D / 512 * ((tiles2 * Hkv + on - 1) / on) + (back ? back_us(pages2.size()) + kJoin : 0);
      };
      int64_t longest = 1;
      double best = 0;
      const int64_t most_steps = ((int64_t)most_len + step - 1) / step;
      const int64_t least = parts_most > 0 ? (most_steps + parts_most - 1) / parts_most : 0;
      const int64_t stride = std::max<int64_t>(1, (most_steps - least) / 256);
      for (int64_t len = std::max<int64_t>(least, 1); len <= most_steps; len += stride) {
        int64_t units = 0;
        for (int32_t g = 0; g < groups->num; ++g) units += pairs_of(g) * ((steps_of(g) + len - 1) / len) * heads;
        const double join = (double)T * Hq * D * ((most_steps + len - 1) / len * 4 + (all_one ? 0 : 4)) / kBytesPerUs;
        for (int32_t on = 0; on <= (all_one && !back ? sms * 3 / 4 : 0); on += 8) {  // SMs left free
          const int64_t clusters = std::max(1, (sms - on) / 2);
          const double parts_us = kCost.start[dx] + (double)((units + clusters - 1) / clusters) *
                                                        ((double)(len * step / 64) * kCost.tile[dx] + kCost.ends[dx]);
          const double cost =
              join + (!all_one ? parts_us : on == 0 ? parts_us + own_us(sms) : std::max(parts_us, own_us(on)));
          if (best == 0 || cost < best) {
            best = cost;
            longest = len;
            p.beside = on;
          }
        }
      }
      // Against every request of a decode step reading its prefix itself, behind the first one's from L2: short
      // prefixes, few requests.
      p.plain = most_len == 0;
      if (all_one) {
        const double n = (double)(tiles * Hkv) / sms, l2 = back ? 0 : (double)(tiles_l2 * Hkv) / sms;
        const double plain =
            kCost.dec_start[cs][dx] +
            (l2 * kCost.dec_l2[cs][dx] + (n - l2) * kCost.dec_dram[cs][dx]) * std::ceil(n) / std::max(n, 1e-9) +
            (back ? back_us((size_t)NP) : 0);
        // (8-bit pools: a page's codes read and its rows written)
        if (set == 1) best += back_us(pre_pages.size());
        p.plain = p.plain || plain <= best + kJoin;
      }
      const int32_t forced = g_test_shared.load(std::memory_order_relaxed);
      if (forced != 0 && most_len > 0) p.plain = forced == 2;
      p.tok.assign((size_t)T, 0);
      std::vector<int32_t> tab, row;
      int32_t pages = 0;  // of the prefixes before
      for (int32_t g = 0; g < groups->num; ++g) {
        const int32_t q0 = qo[groups->indptr[g]], len = tokens_of(g);
        const int64_t few = (steps_of(g) + longest - 1) / longest;
        const int64_t run = few > 0 ? (steps_of(g) + few - 1) / few * step : step;
        const int32_t cut = (int32_t)((pre[g] + run - 1) / run);
        if (!fits_i32((int64_t)cut * T)) return PG_ERR_I32_OVERFLOW;
        for (int32_t i = 0; i < cut; ++i) {
          const int32_t k0 = (int32_t)(i * run), k1 = (int32_t)std::min<int64_t>(k0 + run, pre[g]);
          // (a row stands behind the whole prefix, so it sees every key of the part)
          put_pairs(&tab, cta, q0, len, k1, pages + k0 / ps, pages + (k1 + ps - 1) / ps, k1, k0);
          row.resize(tab.size() / 8, i * T);
        }
        std::fill(p.tok.begin() + q0, p.tok.begin() + q0 + len, cut);
        pages += pre[g] / ps;
      }
      if (!fits_i32((int64_t)(tab.size() / 8) * heads)) return PG_ERR_I32_OVERFLOW;
      p.num = (int32_t)(tab.size() / 8);
      // the longest first, as in the pair table
      std::vector<int32_t> order((size_t)p.num);
      for (int32_t i = 0; i < p.num; ++i) order[i] = i;
      auto keys = [&](int32_t i) { return tab[8 * (size_t)i + 6] - tab[8 * (size_t)i + 7]; };
      std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) { return keys(x) > keys(y); });
      p.tab.assign((size_t)room_parts * 8, 0);
      p.row.assign((size_t)room_parts, 0);
      for (int32_t i = 0; i < p.num; ++i) {
        std::copy_n(tab.data() + 8 * (size_t)order[i], 8, p.tab.data() + 8 * (size_t)i);
        p.row[i] = row[order[i]];
      }
    }
  }
  const int32_t pre_total = (int32_t)pre_pages.size();
  if (groups) {
    pages2.resize((size_t)NP, 0);
    pre_pages.resize((size_t)NP, 0);
    ptab2.resize((size_t)room_pairs * 8, 0);
  }

  // Pack everything into one int32 array and upload it on the plan's stream.
  std::vector<int32_t> host;
  auto put = [&](const int32_t* src, size_t n) {
    const size_t off = host.size();
    host.insert(host.end(), src, src + n);
    while (host.size() % 4) host.push_back(0);  // 16-byte aligned sub-arrays
    return off;
  };
  std::vector<int32_t> tokreq(T);
  for (int32_t r = 0; r < num_req; ++r)
    for (int32_t t = qo[r]; t < qo[r + 1]; ++t) tokreq[t] = r;
  std::vector<int32_t> pids(page_ids, page_ids + NP);

  pg_plan q;
  q.o_live = put(live, 2);
  q.o_qo = put(qo.data(), qo.size());
  q.o_kvp = put(kvp.data(), kvp.size());
  q.o_pages = put(pids.data(), pids.size());
  q.o_last = put(last.data(), last.size());
  q.o_start = put(start.data(), start.size());
  q.o_kvs = put(kvs.data(), kvs.size());
  q.o_tokreq = put(tokreq.data(), tokreq.size());
  q.o_wreq = put(wreq.data(), wreq.size());
  q.o_wtok = put(wtok.data(), wtok.size());
  q.o_pair = put(ptab.data(), ptab.size());
  std::unique_ptr<pg_plan> own;
  if (groups) {
    own.reset(new pg_plan);
    own->o_live = q.o_live;
    own->o_qo = q.o_qo;
    own->o_last = q.o_last;
    own->o_start = q.o_start;
    own->o_tokreq = q.o_tokreq;
    own->o_wreq = q.o_wreq;
    own->o_wtok = q.o_wtok;
    own->o_kvp = put(kvp2.data(), kvp2.size());
    own->o_pages = put(pages2.data(), pages2.size());
    own->o_kvs = put(kvs2.data(), kvs2.size());
    own->o_pair = put(ptab2.data(), ptab2.size());
    for (int set = 0; set < 2; ++set) {
      const Parts& p = parts[set];
      const int32_t count[3] = {0, p.num, pre_total};
      q.parts[set] = PartSet{p.num, p.beside, p.plain, put(p.tab.data(), p.tab.size()), put(p.row.data(), p.row.size()),
                             put(count, 3), put(p.tok.data(), p.tok.size())};
    }
    q.o_pre_pages = put(pre_pages.data(), pre_pages.size());
  }
  if (host.empty()) host.assign(4, 0);

  int err = PG_OK;
  if (!status_word(&err)) return err;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PG_ERR_CUDA;
  // the upload goes through this plan's next pinned staging buffer (see PlanStage)
  PlanStage& st = p->stage;
  const int k = st.next;
  const size_t bytes = host.size() * sizeof(int32_t);
  if (!st.done[k]) {
    if (cudaEventCreateWithFlags(&st.done[k], cudaEventDisableTiming) != cudaSuccess) {
      st.done[k] = nullptr;
      return PG_ERR_CUDA;
    }
  } else if (cudaEventSynchronize(st.done[k]) != cudaSuccess) {
    return PG_ERR_CUDA;
  }
  if (st.cap[k] < bytes) {
    if (st.host[k]) cudaFreeHost(st.host[k]);
    st.host[k] = nullptr;
    st.cap[k] = 0;
    if (cudaMallocHost((void**)&st.host[k], bytes) != cudaSuccess) {
      st.host[k] = nullptr;
      return PG_ERR_CUDA;
    }
    st.cap[k] = bytes;
  }
  std::memcpy(st.host[k], host.data(), bytes);
  // An existing plan whose device storage is large enough is updated in place: the copy is
  // ordered on the plan's stream after every call already queued with the old metadata (a plan
  // is used on its own stream only), and a CUDA graph that captured the plan keeps reading live
  // metadata. Otherwise new storage is allocated and the old freed after the commit.
  int32_t* d = nullptr;
  const bool fresh = !(p->dev && p->dev_cap >= bytes);
  if (fresh) {
    if (cudaMallocAsync((void**)&d, bytes, stream) != cudaSuccess) return PG_ERR_CUDA;
  } else {
    d = p->dev;
  }
  if (cudaMemcpyAsync(d, st.host[k], bytes, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
      cudaEventRecord(st.done[k], stream) != cudaSuccess) {
    if (fresh) cudaFreeAsync(d, stream);
    return PG_ERR_CUDA;
  }
  st.next = k ^ 1;

  q.num_req = num_req; q.num_tokens = T; q.num_qo_heads = Hq; q.num_kv_heads = Hkv;
  q.head_dim = D; q.page_size = ps;
  q.max_page_id = max_page; q.max_last_page_len = max_last; q.max_qo_len = max_qo;
  q.max_kv_len = max_kv; q.max_pos_end = max_end;
  q.cta_tile_q = cta; q.decode = all_one ? 1 : 0; q.kv_chunk = chunk;
  // decode partials: a query sees at most window + 1 keys in ring addressing
  const int64_t seen = ring ? std::min<int64_t>(max_kv, (int64_t)ring_window + 1) : max_seen;
  q.max_chunks = seen > 0 ? (int32_t)((seen + chunk - 1) / chunk) : 0;
  q.ring = ring ? 1 : 0;
  q.ring_window = ring ? ring_window : -1;
  q.segment = segment ? 1 : 0;
  q.prep_ok = prep_ok ? 1 : 0;
  q.num_work = (int32_t)nwork; q.num_pairs = npairs; q.num_page_ids = NP;
  q.room_work = room_work; q.room_pairs = room_pairs;
  q.stream = stream; q.device = dev;
  q.dev = d; q.dev_elems = host.size();
  q.dev_cap = fresh ? bytes : p->dev_cap;
  q.max_seen = max_seen;
  q.page_keys = num_req > 0 ? (int32_t)std::min<int64_t>((int64_t)(NP - num_req + 1) * ps, INT32_MAX) : 0;
  q.tiles = tiles;
  q.host_ids = std::move(pids);
  if (groups) {
    auto fields = [](pg_plan* o, const pg_plan& f) {
      o->num_req = f.num_req; o->num_tokens = f.num_tokens; o->num_qo_heads = f.num_qo_heads;
      o->num_kv_heads = f.num_kv_heads; o->head_dim = f.head_dim; o->page_size = f.page_size;
      o->max_page_id = f.max_page_id; o->max_last_page_len = f.max_last_page_len; o->max_qo_len = f.max_qo_len;
      o->max_kv_len = f.max_kv_len; o->max_pos_end = f.max_pos_end; o->cta_tile_q = f.cta_tile_q;
      o->decode = f.decode; o->kv_chunk = f.kv_chunk; o->num_work = f.num_work; o->num_pairs = f.num_pairs;
      o->room_work = f.room_work; o->room_pairs = f.room_pairs; o->stream = f.stream; o->device = f.device;
      o->dev = f.dev; o->dev_elems = f.dev_elems; o->dev_cap = f.dev_cap;
    };
    fields(own.get(), q);
    own->segment = 1;
    own->max_chunks = (seen2 + chunk - 1) / chunk;
    own->num_page_ids = NP;  // (the list's room: a captured call covers whatever an update leaves in it)
    own->max_seen = seen2;
    own->page_keys = num_req > 0 ? (int32_t)std::min<int64_t>((int64_t)(NP - num_req + 1) * ps, INT32_MAX) : 0;
    own->tiles = tiles2;
    q.own = std::move(own);
    q.num_groups = groups->num;
    q.room_parts = room_parts;
    q.parts_most = parts_most;
    q.prefix_pages = pre_total;
  }

  // Commit: only now does the caller's plan change.
  int32_t* old = p->dev;
  q.stage = p->stage;
  *p = std::move(q);
  if (fresh && old) cudaFreeAsync(old, stream);
  return PG_OK;
}

PlanDev plan_dev(const pg_plan* p) {
  PlanDev v;
  v.qo_indptr = p->dev + p->o_qo;
  v.kv_page_indptr = p->dev + p->o_kvp;
  v.page_ids = p->dev + p->o_pages;
  v.last_page_len = p->dev + p->o_last;
  v.start_pos = p->dev + p->o_start;
  v.kv_start = p->dev + p->o_kvs;
  v.tok_req = p->dev + p->o_tokreq;
  v.work_req = p->dev + p->o_wreq;
  v.work_tok0 = p->dev + p->o_wtok;
  v.pair_tab = p->dev + p->o_pair;
  v.num_req = p->num_req;
  v.num_tokens = p->num_tokens;
  v.num_page_ids = p->num_page_ids;
  v.num_work = p->num_work;
  v.num_pairs = p->num_pairs;
  v.ring = p->ring;
  v.live = nullptr;
  return v;
}

// A captured launch is replayed under plans that are updated in place: what it bakes in has to hold
// for any plan of as many requests, tokens and pages.
bool capturing(cudaStream_t stream) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &st) != cudaSuccess) {
    cudaGetLastError();  // (the legacy stream beside another stream's capture: the launch reports it)
    return false;
  }
  return st == cudaStreamCaptureStatusActive;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// checked_paged_geometry: the pool descriptor must be self-consistent for head_dim D.
int check_pool(const pg_pool_t* pool, int32_t D) {
  if (!pool || !pool->base) return PG_ERR_ARG;
  if (pool->head_dim != D) return PG_ERR_LAYOUT;
  if (pool->num_layers <= 0 || pool->num_pages <= 0 || pool->page_size <= 0 ||
      pool->num_kv_heads <= 0)
    return PG_ERR_LAYOUT;
  if (!aligned16(pool->base)) return PG_ERR_ALIGN;
  int64_t s_slot = D, s_head, s_kv, s_page, s_layer, total;
  if (!mul_i64(pool->page_size, s_slot, &s_head) || !mul_i64(pool->num_kv_heads, s_head, &s_kv) ||
      !mul_i64(2, s_kv, &s_page) || !mul_i64(pool->num_pages, s_page, &s_layer) ||
      !mul_i64(pool->num_layers, s_layer, &total))
    return PG_ERR_I32_OVERFLOW;
  if (pool->stride_slot != s_slot || pool->stride_head != s_head || pool->stride_kv != s_kv ||
      pool->stride_page != s_page || pool->stride_layer != s_layer)
    return PG_ERR_LAYOUT;
  if (pool->capacity != total) return PG_ERR_LAYOUT;  // whole pages, every layer
  return PG_OK;
}

// Plan vs pool agreement plus the recorded page bounds, before every launch.
int check_plan_pool(const pg_plan* p, const pg_pool_t* pool, int32_t layer, int32_t D) {
  if (p->head_dim != D) return PG_ERR_PLAN_MISMATCH;
  int rc = check_pool(pool, D);
  if (rc) return rc;
  if (p->num_kv_heads != pool->num_kv_heads || p->page_size != pool->page_size)
    return PG_ERR_PLAN_MISMATCH;
  if (layer < 0 || layer >= pool->num_layers) return PG_ERR_LAYER;
  if (p->max_page_id >= pool->num_pages) return PG_ERR_PAGE_OOB;
  if (p->max_last_page_len > pool->page_size) return PG_ERR_LAST_PAGE_LEN;
  return PG_OK;
}

PoolDev pool_dev(const pg_pool_t* pool, int32_t layer) {
  PoolDev v;
  v.layer_base = reinterpret_cast<__nv_bfloat16*>(pool->base) + (int64_t)layer * pool->stride_layer;
  v.stride_page = pool->stride_page;
  v.stride_kv = pool->stride_kv;
  v.stride_head = pool->stride_head;
  v.num_pages = pool->num_pages;
  v.page_size = pool->page_size;
  v.num_kv_heads = pool->num_kv_heads;
  v.head_dim = pool->head_dim;
  return v;
}

// ---- 8-bit pools
int check_q8(const pg_q8_pool_t* pool, int32_t D) {
  if (!pool || !pool->codes || !pool->scales) return PG_ERR_ARG;
  if (pool->head_dim != D) return PG_ERR_LAYOUT;
  if (pool->num_layers <= 0 || pool->num_pages <= 0 || pool->page_size <= 0 || pool->num_kv_heads <= 0)
    return PG_ERR_LAYOUT;
  if (!aligned16(pool->codes)) return PG_ERR_ALIGN;
  int64_t rows = 0, codes = 0;
  if (!mul_i64((int64_t)pool->num_layers * 2, pool->num_pages, &rows) ||
      !mul_i64(rows, pool->num_kv_heads, &rows) || !mul_i64(rows, pool->page_size, &rows) ||
      !mul_i64(rows, D, &codes) || !mul_i64(codes, 2, &codes))
    return PG_ERR_I32_OVERFLOW;
  return pool->capacity == rows ? PG_OK : PG_ERR_LAYOUT;
}
int check_plan_q8(const pg_plan* p, const pg_q8_pool_t* pool, int32_t layer, int32_t num_layers) {
  if (p->head_dim != 256 && p->head_dim != 512) return PG_ERR_PLAN_MISMATCH;
  int rc = check_q8(pool, p->head_dim);
  if (rc) return rc;
  if (p->num_kv_heads != pool->num_kv_heads || p->page_size != pool->page_size) return PG_ERR_PLAN_MISMATCH;
  if (layer < 0 || num_layers < 1 || layer > pool->num_layers - num_layers) return PG_ERR_LAYER;
  return p->max_page_id >= pool->num_pages ? PG_ERR_PAGE_OOB : PG_OK;
}
Q8Dev q8_dev(const pg_q8_pool_t* pool, int32_t layer) {
  Q8Dev v;
  v.rows_layer = (int64_t)pool->num_pages * 2 * pool->num_kv_heads * pool->page_size;
  v.codes = pool->codes + layer * v.rows_layer * pool->head_dim;
  v.scales = pool->scales + layer * v.rows_layer;
  return v;
}
// The geometry as kernels read it; strides in elements (codes), no storage.
PoolDev q8_geometry(const pg_q8_pool_t* pool) {
  PoolDev v{};
  v.num_pages = pool->num_pages;
  v.page_size = pool->page_size;
  v.num_kv_heads = pool->num_kv_heads;
  v.head_dim = pool->head_dim;
  v.stride_head = (int64_t)pool->page_size * pool->head_dim;
  v.stride_kv = pool->num_kv_heads * v.stride_head;
  v.stride_page = 2 * v.stride_kv;
  return v;
}

int check_tok_input(const pg_bf16_t* p, int64_t stride, int32_t heads, int32_t D) {
  if (!p) return PG_ERR_ARG;
  if (stride < (int64_t)heads * D) return PG_ERR_ARG;
  if (!aligned16(p) || stride % 8 != 0) return PG_ERR_ALIGN;
  return PG_OK;
}

// The geometry checks of a prep call's pool, and its device view.
struct PrepPool {
  const pg_pool_t* bf16;
  const pg_q8_pool_t* q8;
};
int check_prep_pool(const pg_plan* plan, const PrepPool& p, int32_t layer, int32_t D) {
  return p.q8 ? check_plan_q8(plan, p.q8, layer, 1) : check_plan_pool(plan, p.bf16, layer, D);
}

int prep_common(const pg_plan* plan, const PrepPool& pool, int32_t layer, int32_t D,
                const pg_bf16_t* q_raw, int64_t qs, const pg_bf16_t* k_raw, int64_t ks,
                const pg_bf16_t* v_raw, int64_t vs, const pg_bf16_t* w_q, const pg_bf16_t* w_k,
                float eps, const float* rc, const float* rsn, int32_t rope_rows,
                pg_bf16_t* q_out, cudaStream_t stream, PrepArgs* a) {
  if (!plan) return PG_ERR_ARG;
  if (stream != plan->stream) return PG_ERR_STREAM;
  // a key-segment plan takes prep only when every step's tokens are its segment's tail
  if (plan->segment && !plan->prep_ok) return PG_ERR_COVERAGE;
  int rc_ = check_prep_pool(plan, pool, layer, D);
  if (rc_) return rc_;
  if (!std::isfinite(eps) || !(eps > 0.0f)) return PG_ERR_NONFINITE;
  if (plan->num_tokens == 0) return PG_OK;
  if (!rc || !rsn || !w_q || !w_k || !q_out) return PG_ERR_ARG;
  if (rope_rows < 1) return PG_ERR_ARG;
  if (plan->max_pos_end > rope_rows) return PG_ERR_ROPE_RANGE;
  if ((rc_ = check_tok_input(q_raw, qs, plan->num_qo_heads, D))) return rc_;
  if ((rc_ = check_tok_input(k_raw, ks, plan->num_kv_heads, D))) return rc_;
  if (D == 256 && (rc_ = check_tok_input(v_raw, vs, plan->num_kv_heads, D))) return rc_;
  if (!aligned16(w_q) || !aligned16(w_k) || !aligned16(q_out) || !aligned16(rc) || !aligned16(rsn))
    return PG_ERR_ALIGN;
  int64_t span = 0;  // largest element offset any raw input row reaches must fit int64
  if (!mul_i64((int64_t)plan->num_tokens, qs > ks ? (qs > vs ? qs : vs) : (ks > vs ? ks : vs), &span))
    return PG_ERR_I32_OVERFLOW;
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  a->plan = plan_dev(plan);
  if (pool.q8) {
    a->pool = q8_geometry(pool.q8);
    a->q8 = q8_dev(pool.q8, layer);
  } else {
    a->pool = pool_dev(pool.bf16, layer);
    a->q8 = Q8Dev{};
  }
  a->q_raw = reinterpret_cast<const __nv_bfloat16*>(q_raw);
  a->k_raw = reinterpret_cast<const __nv_bfloat16*>(k_raw);
  a->v_raw = reinterpret_cast<const __nv_bfloat16*>(v_raw);
  a->q_stride = qs; a->k_stride = ks; a->v_stride = vs;
  a->w_q = reinterpret_cast<const __nv_bfloat16*>(w_q);
  a->w_k = reinterpret_cast<const __nv_bfloat16*>(w_k);
  a->rope_cos = rc; a->rope_sin = rsn;
  a->q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  a->eps = eps;
  a->rope_rows = rope_rows;
  a->num_qo_heads = plan->num_qo_heads;
  a->status = st;
  return PG_OK;
}

size_t workspace_bytes(const pg_plan* p) {
  if (!p || !p->decode || p->num_req == 0) return 0;
  const int32_t group = p->num_qo_heads / p->num_kv_heads;
  if (attn_decode_stream_supported(p->head_dim, group, p->page_size))
    return attn_decode_stream_ws_bytes(p->num_req, group, p->head_dim);
  const size_t rows = (size_t)p->num_req * p->num_qo_heads * p->max_chunks;
  return rows * (size_t)p->head_dim * sizeof(float) + rows * 2 * sizeof(float);
}

// Bounded-cache attention: the sinks, and the decode scores to keep (see AttnArgs).
struct Bounded {
  int32_t num_sink = 0;
  float* logits = nullptr;
  int64_t logit_slots = 0;
  StatsDev stats = {};
  bool in_order = false;              // the pool's pages lie in the order of the plan's list
  const AttnArgs* parts = nullptr;    // decode: parts of the rows' prefixes, for the join
};
// The parts' records into the arguments of the call on the own keys.
void take_parts(AttnArgs* a, const AttnArgs* parts) {
  if (!parts) return;
  a->part_o = parts->part_o;
  a->part_ml = parts->part_ml;
  a->tok_parts = parts->tok_parts;
  a->join_lse = parts->join_lse;
  a->beside = parts->beside;
}

int32_t plan_max_tiles(const pg_plan* p) {
  return (int32_t)std::min<int64_t>(p->tiles * p->num_kv_heads, INT32_MAX);
}
// Bytes of one chunk's partials over all rows of a decode step.
size_t chunk_bytes(const pg_plan* p) {
  return (size_t)p->num_req * p->num_qo_heads * ((size_t)p->head_dim + 2) * sizeof(float);
}
// Chunks per request of the bounded-cache form's chunked kernel: the plan's, as far as they fit the
// workspace of the entries that take no sinks (where those run the streaming kernel, whose records
// do not grow with the keys; longer chunks make up for it, and a single one leaves no partials).
int32_t bounded_chunks(const pg_plan* p) {
  return (int32_t)std::min<size_t>(p->max_chunks, std::max<size_t>(1, workspace_bytes(p) / chunk_bytes(p)));
}
bool bounded_tc(const pg_plan* p) {
  return bounded_decode_supported(p->head_dim, p->num_qo_heads / p->num_kv_heads, p->page_size);
}
// Workspace of the bounded-cache form: the tensor-core kernel's records for every CTA (it does with
// fewer), or the chunked kernel's partials where that one runs.
size_t bounded_ws_bytes(const pg_plan* p) {
  if (!p || !p->decode || p->num_req == 0) return 0;
  if (bounded_tc(p))
    return bounded_decode_ws_bytes(p->num_req, p->num_qo_heads / p->num_kv_heads, p->head_dim, plan_max_tiles(p));
  const int32_t chunks = bounded_chunks(p);
  return chunks > 1 ? chunks * chunk_bytes(p) : 0;
}

// Geometry, window and scale of an attention call.
int check_attn_args(const pg_plan* plan, int32_t D, int32_t window_left, float sm_scale) {
  const int32_t group = plan->num_qo_heads / plan->num_kv_heads;
  const int32_t kernel_cta = attn_kernel_cta_tile_q(D, group, plan->page_size);
  if (kernel_cta == 0 || kernel_cta != plan->cta_tile_q) return PG_ERR_PLAN_MISMATCH;
  if (attn_kernel_kv_chunk(D) != plan->kv_chunk) return PG_ERR_PLAN_MISMATCH;
  if (window_left < -1) return PG_ERR_WINDOW;
  // ring addressing holds only the window the plan was built for
  if (plan->ring && (window_left < 0 || window_left > plan->ring_window)) return PG_ERR_WINDOW;
  if (!std::isfinite(sm_scale)) return PG_ERR_NONFINITE;
  // the chunked decode kernel's grid holds the key chunks of a request in its z dimension
  if (plan->decode && !attn_decode_stream_supported(D, group, plan->page_size) &&
      plan->max_chunks > 65535)
    return PG_ERR_I32_OVERFLOW;
  return PG_OK;
}
// The rows that an attention call reads and writes.
int check_attn_rows(const pg_bf16_t* q, const pg_bf16_t* out, const float* lse) {
  if (!q || !out) return PG_ERR_ARG;
  // the tensor-core prefill kernel reads Q rows and writes output rows in 32-byte accesses
  if ((((uintptr_t)q | (uintptr_t)out) & 31u) != 0) return PG_ERR_ALIGN;
  return lse && ((uintptr_t)lse & 3u) != 0 ? PG_ERR_ALIGN : PG_OK;
}

// `args` (the accumulating entry, whose workspace holds more) receives the launched call's
// arguments, with num_tokens 0 when nothing ran.
int attn_common(const pg_plan* plan, const pg_pool_t* pool, int32_t layer, int32_t D,
                const pg_bf16_t* q, pg_bf16_t* out, float* lse, int32_t window_left,
                float sm_scale, void* ws, size_t ws_bytes, cudaStream_t stream,
                const Bounded* bounded = nullptr, AttnArgs* args = nullptr) {
  if (args) args->plan.num_tokens = 0;
  if (!plan) return PG_ERR_ARG;
  if (stream != plan->stream) return PG_ERR_STREAM;
  const bool listed = bounded && bounded->in_order;
  int rc = listed ? check_pool(pool, D) : check_plan_pool(plan, pool, layer, D);
  if (rc) return rc;
  if ((rc = check_attn_args(plan, D, window_left, sm_scale))) return rc;
  const int32_t group = plan->num_qo_heads / plan->num_kv_heads;
  const bool tma_rows = plan->decode ? attn_decode_stream_supported(D, group, plan->page_size)
                                     : attn_tc_supported(D, group, plan->page_size);
  if (tma_rows && (int64_t)pool->num_pages * 2 * pool->num_kv_heads * pool->page_size > INT32_MAX)
    return PG_ERR_I32_OVERFLOW;  // tensor-map row coordinates are int32
  if (plan->num_tokens == 0) return PG_OK;
  if ((rc = check_attn_rows(q, out, lse))) return rc;
  const size_t need = args ? bounded_ws_bytes(plan) : workspace_bytes(plan);
  if (need > 0) {
    if (!ws || ws_bytes < need) return PG_ERR_WORKSPACE;
    if (!aligned16(ws)) return PG_ERR_ALIGN;
  }
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  AttnArgs a;
  a.plan = plan_dev(plan);
  if (!plan->decode && capturing(stream)) {
    a.plan.live = plan->dev + plan->o_live;
    a.plan.num_work = plan->room_work;
    a.plan.num_pairs = plan->room_pairs;
  }
  if (listed) a.plan.page_ids = nullptr;
  a.pool = pool_dev(pool, layer);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  a.window_left = window_left;
  a.num_qo_heads = plan->num_qo_heads;
  a.group = group;
  a.cta_tile_q = plan->cta_tile_q;
  a.kv_chunk = plan->kv_chunk;
  a.max_chunks = plan->max_chunks;
  a.status = st;
  a.bounded = bounded ? 1 : 0;
  a.bounded_chunks = bounded && plan->decode ? bounded_chunks(plan) : 0;
  a.num_sink = bounded ? bounded->num_sink : 0;
  a.logits = bounded ? bounded->logits : nullptr;
  a.logit_slots = bounded ? bounded->logit_slots : 0;
  a.stats = bounded ? bounded->stats : StatsDev{};
  a.max_keys = plan->max_seen;
  a.max_tiles = plan_max_tiles(plan);
  wait_settings(&a.wait_ns, &a.test_withhold);
  cudaError_t e;
  a.ws_raw = ws;
  a.ws_bytes = ws_bytes;
  a.ws_o = nullptr;
  a.ws_ml = nullptr;
  if (bounded) take_parts(&a, bounded->parts);
  if (args) *args = a;
  if (plan->decode) {
    e = launch_attn_decode(a, D, stream);
  } else {
    e = launch_attn_prefill(a, D, stream);
  }
  return e == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

// ---- bounded-cache operators: checks shared by their entries
// A page that two places of the page list name has no statistics of its own, and rows moved
// within it for one request would move under the other.
int shares_pages(const pg_plan* p, bool* out) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  if (p->shared < 0) {
    try {
      // one bit per page, or a sort where the page ids are far sparser than that
      bool twice = false;
      const size_t words = (size_t)(p->max_page_id + 1) / 64 + 1;
      if (words <= p->host_ids.size() + 4096) {
        std::vector<uint64_t> seen(words, 0);
        for (const int32_t id : p->host_ids) {
          const uint64_t bit = 1ull << (id & 63);
          twice |= (seen[id >> 6] & bit) != 0;
          seen[id >> 6] |= bit;
        }
      } else {
        std::vector<int32_t> ids(p->host_ids);
        std::sort(ids.begin(), ids.end());
        twice = std::adjacent_find(ids.begin(), ids.end()) != ids.end();
      }
      p->shared = twice ? 1 : 0;
    } catch (const std::bad_alloc&) {
      return PG_ERR_ARG;
    }
  }
  *out = p->shared == 1;
  return PG_OK;
}

int check_stats(const pg_plan* p, const pg_kv_stats_t* st, int32_t layer, int32_t num_layers) {
  if (!st || !st->mass || !st->pos) return PG_ERR_ARG;
  if (st->num_layers <= 0 || st->num_pages <= 0 || st->page_size <= 0 || st->num_kv_heads <= 0)
    return PG_ERR_LAYOUT;
  if (((uintptr_t)st->mass & 3u) || ((uintptr_t)st->pos & 3u)) return PG_ERR_ALIGN;
  int64_t n = 0;
  if (!mul_i64(st->num_layers, st->num_pages, &n) || !mul_i64(n, st->num_kv_heads, &n) ||
      !mul_i64(n, st->page_size, &n))
    return PG_ERR_I32_OVERFLOW;
  if (st->capacity != n) return PG_ERR_LAYOUT;
  if (p->num_kv_heads != st->num_kv_heads || p->page_size != st->page_size)
    return PG_ERR_PLAN_MISMATCH;
  if (layer < 0 || num_layers < 1 || layer > st->num_layers - num_layers) return PG_ERR_LAYER;
  if (p->max_page_id >= st->num_pages) return PG_ERR_PAGE_OOB;
  return PG_OK;
}

StatsDev stats_dev(const pg_kv_stats_t* st, int32_t layer) {
  StatsDev v;
  v.stride_layer = (int64_t)st->num_pages * st->num_kv_heads * st->page_size;
  v.mass = st->mass + layer * v.stride_layer;
  v.pos = st->pos + layer * v.stride_layer;
  return v;
}

// plan, stream and device of a bounded-cache call
int check_bounded_plan(const pg_plan* plan, cudaStream_t stream) {
  if (!plan) return PG_ERR_ARG;
  if (stream != plan->stream) return PG_ERR_STREAM;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PG_ERR_CUDA;
  if (dev != plan->device) return PG_ERR_STREAM;
  if (plan->ring) return PG_ERR_PLAN_MISMATCH;  // a ring overwrites the positions these keep
  return PG_OK;
}

// The attention kernels count keys in tiles, so a position past the step's last one by less than a
// pair of query tiles (256 rows) and a key tile (128) must still be an int32.
constexpr int32_t kLastEnd = INT32_MAX - 1024;
int check_bounded_attn(const pg_plan* plan, int32_t num_sink) {
  if (num_sink < 0) return PG_ERR_WINDOW;
  if (plan->head_dim != 256 && plan->head_dim != 512) return PG_ERR_PLAN_MISMATCH;
  return plan->max_pos_end > kLastEnd ? PG_ERR_I32_OVERFLOW : PG_OK;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Scores that a decode step of the plan keeps: [slots of the page list][num_qo_heads].
int64_t logit_slots(const pg_plan* p) { return (int64_t)p->num_page_ids * p->page_size; }

bool mass_on_tensor_cores(const pg_plan* p) {
  return !p->decode && p->num_req > 0 &&
         attn_tc_supported(p->head_dim, p->num_qo_heads / p->num_kv_heads, p->page_size);
}
size_t mass_workspace_bytes(const pg_plan* p) {
  if (!p || p->num_req == 0) return 0;
  if (p->decode)
    return align256(bounded_ws_bytes(p)) + (size_t)logit_slots(p) * p->num_qo_heads * sizeof(float);
  return mass_on_tensor_cores(p) ? mass_tc_ws_bytes() : 0;
}

// Checks of an eviction call, and its arguments.
int evict_common(const pg_plan* plan, const pg_kv_stats_t* stats, int32_t layer, int32_t num_layers,
                 int32_t budget, const int32_t* src, cudaStream_t stream, EvictArgs* a) {
  int rc = check_bounded_plan(plan, stream);
  if (rc) return rc;
  if ((rc = check_stats(plan, stats, layer, num_layers))) return rc;
  if (budget < 1) return PG_ERR_ARG;
  bool shared = false;
  if ((rc = shares_pages(plan, &shared))) return rc;
  if (shared) return PG_ERR_SHARED_PAGE;
  a->plan = plan_dev(plan);
  if (plan->num_req == 0) return PG_OK;
  if (!src) return PG_ERR_ARG;
  if ((uintptr_t)src & 3u) return PG_ERR_ALIGN;
  // every grid of the call fits
  int64_t segs = 0, blocks = 0;
  // (slots of the budget that no request fills hold -1: they need no block of apply)
  a->slots = std::min(capturing(stream) ? plan->page_keys : plan->max_seen, budget);
  const int32_t per_seg = std::max(evict_select_ranks(plan->max_seen), evict_apply_blocks(a->slots));
  if (!mul_i64(num_layers, plan->num_req, &segs) || !mul_i64(segs, plan->num_kv_heads, &segs) ||
      !mul_i64(segs, per_seg, &blocks) || !fits_i32(segs) || !fits_i32(blocks))
    return PG_ERR_I32_OVERFLOW;
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  a->pool = PoolDev{};
  a->pool.num_pages = stats->num_pages;
  a->pool.page_size = stats->page_size;
  a->pool.num_kv_heads = stats->num_kv_heads;
  a->pool.head_dim = plan->head_dim;
  a->pool_stride_layer = 0;
  a->stats = stats_dev(stats, layer);
  a->src = const_cast<int32_t*>(src);
  a->num_layers = num_layers;
  a->budget = budget;
  a->num_sink = a->num_recent = 0;
  a->max_keys = plan->max_seen;
  set_page_divisor(a);
  a->status = st;
  return PG_OK;
}

// ---- attention over an 8-bit cache
size_t align1k(size_t n) { return (n + 1023) & ~(size_t)1023; }

// Plans that the 8-bit kernels do not take are read back first: the workspace holds the pages in the
// order of the plan's list, and what the bf16 kernel needs. (No list of them: a decode kernel looks at
// page ids while the stream's previous kernel, which would have written it, still runs.)
struct ReadBack {
  size_t rest, bytes;  // offset of the kernel's workspace, total
};
bool read_back(const pg_plan* p, ReadBack* w) {
  const __int128 page = (__int128)4 * p->num_kv_heads * p->page_size * p->head_dim;
  const __int128 pages = page * p->num_page_ids;
  if (pages > ((__int128)1 << 60)) return false;
  w->rest = align1k((size_t)pages);
  w->bytes = w->rest + std::max(workspace_bytes(p), bounded_ws_bytes(p));
  return true;
}
bool q8_direct(const pg_plan* p) {
  return p->decode && q8_decode_supported(p->head_dim, p->num_qo_heads / p->num_kv_heads, p->page_size);
}
size_t q8_workspace_bytes(const pg_plan* p) {
  if (!p || p->num_req == 0 || (p->head_dim != 256 && p->head_dim != 512)) return 0;
  if (q8_direct(p))
    return q8_decode_ws_bytes(p->num_req, p->num_qo_heads / p->num_kv_heads, p->head_dim, plan_max_tiles(p));
  ReadBack w;
  return read_back(p, &w) ? w.bytes : SIZE_MAX;
}

int q8_attn(const pg_plan* plan, const pg_q8_pool_t* pool, int32_t layer, const pg_bf16_t* q, pg_bf16_t* out,
            float* lse, int32_t window_left, int32_t num_sink, float sm_scale, void* ws, size_t ws_bytes,
            cudaStream_t stream, const AttnArgs* parts = nullptr) {
  int rc = check_bounded_plan(plan, stream);
  if (rc || (rc = check_bounded_attn(plan, num_sink))) return rc;
  if ((rc = check_plan_q8(plan, pool, layer, 1))) return rc;
  const int32_t D = plan->head_dim;
  // what the bf16 call would refuse is refused before the read-back is launched
  if ((rc = check_attn_args(plan, D, window_left, sm_scale))) return rc;
  const bool direct = q8_direct(plan);
  if ((int64_t)(direct ? pool->num_pages : plan->num_page_ids) * 2 * plan->num_kv_heads * plan->page_size > INT32_MAX)
    return PG_ERR_I32_OVERFLOW;  // tensor-map row coordinates are int32
  if (plan->num_tokens == 0) return PG_OK;
  if ((rc = check_attn_rows(q, out, lse))) return rc;
  if (direct) {
    if (!ws || ws_bytes < q8_workspace_bytes(plan)) return PG_ERR_WORKSPACE;
    if (!aligned16(ws)) return PG_ERR_ALIGN;
    int err = PG_OK;
    AttnArgs a{};
    if (!(a.status = status_word(&err))) return err;
    a.plan = plan_dev(plan);
    a.pool = q8_geometry(pool);
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.ws_raw = ws;
    a.ws_bytes = ws_bytes;
    a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    a.window_left = window_left;
    a.num_sink = num_sink;
    a.num_qo_heads = plan->num_qo_heads;
    a.group = plan->num_qo_heads / plan->num_kv_heads;
    a.bounded = 1;
    a.max_keys = plan->max_seen;
    a.max_tiles = plan_max_tiles(plan);
    wait_settings(&a.wait_ns, &a.test_withhold);
    take_parts(&a, parts);
    return launch_q8_decode(a, q8_dev(pool, layer), D, stream) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
  }
  ReadBack w;
  if (!read_back(plan, &w) || !ws || ws_bytes < w.bytes) return PG_ERR_WORKSPACE;
  if (!aligned16(ws)) return PG_ERR_ALIGN;
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  unsigned char* const base = static_cast<unsigned char*>(ws);
  DequantArgs d{};
  d.plan = plan_dev(plan);
  d.src = q8_dev(pool, layer);
  d.dst = reinterpret_cast<__nv_bfloat16*>(base);
  d.num_pages = pool->num_pages;
  d.page_size = plan->page_size;
  d.num_kv_heads = plan->num_kv_heads;
  d.head_dim = D;
  d.num_layers = 1;
  d.list = 1;
  d.window_left = window_left;
  d.num_sink = num_sink;
  d.status = st;
  if (launch_dequant(d, stream) != cudaSuccess) return PG_ERR_CUDA;
  const int32_t ps = plan->page_size, H = plan->num_kv_heads;
  const pg_pool_t copy = {reinterpret_cast<pg_bf16_t*>(base), 1, plan->num_page_ids, ps, H, D,
                          (int64_t)plan->num_page_ids * 2 * H * ps * D, (int64_t)2 * H * ps * D,
                          (int64_t)H * ps * D, (int64_t)ps * D, D, (int64_t)plan->num_page_ids * 2 * H * ps * D};
  Bounded b;
  b.num_sink = num_sink;
  b.in_order = true;
  return attn_common(plan, &copy, 0, D, q, out, lse, window_left, sm_scale, base + w.rest, ws_bytes - w.rest, stream,
                     &b);
}

// ---- attention over shared prefixes
// The workspace: the parts' records, the rows' lse, and what the call on the own keys needs.
struct SharedWs {
  size_t ml, o, lse, own, bytes;
};
bool shared_ws(const pg_plan* p, size_t own_bytes, SharedWs* w) {
  const __int128 rows = (__int128)p->num_tokens * p->num_qo_heads, recs = rows * p->parts_most;
  if (recs * p->head_dim * 4 > ((__int128)1 << 60)) return false;
  w->ml = 0;
  w->o = align256((size_t)recs * 2 * sizeof(float));
  w->lse = w->o + align256((size_t)recs * p->head_dim * sizeof(float));
  w->own = w->lse + align256((size_t)rows * sizeof(float));
  w->bytes = w->own + own_bytes;
  return true;
}
// A workspace is 16-byte aligned, the records 256: the offsets count from here.
constexpr size_t kSharedPad = 256;
unsigned char* shared_base(void* ws) {
  return reinterpret_cast<unsigned char*>(((uintptr_t)ws + kSharedPad - 1) & ~(uintptr_t)(kSharedPad - 1));
}
size_t shared_workspace_bytes(const pg_plan* p) {
  if (!p || !p->own || p->num_req == 0) return 0;
  SharedWs w;
  if (!shared_ws(p, std::max(workspace_bytes(p->own.get()), bounded_ws_bytes(p->own.get())), &w)) return SIZE_MAX;
  // (enough for the plain walk: an update may take either)
  return std::max(w.bytes + kSharedPad, std::max(workspace_bytes(p), bounded_ws_bytes(p)));
}

// The prefixes' parts: pool pages `page_ids` (device, prefix by prefix; null: in that order) of `pool`.
AttnArgs part_args(const pg_plan* p, const PartSet& set, const PoolDev& pool, const int32_t* page_ids,
                   int32_t num_page_ids, const pg_bf16_t* q, float sm_scale, unsigned char* base, const SharedWs& w, int* status) {
  AttnArgs a{};
  a.plan = plan_dev(p);
  a.plan.pair_tab = p->dev + set.o_tab;
  a.plan.page_ids = page_ids;
  a.plan.num_page_ids = num_page_ids;
  a.plan.num_pairs = set.num;
  if (capturing(p->stream)) {
    a.plan.live = p->dev + set.o_live;
    a.plan.num_pairs = p->room_parts;
  }
  a.pool = pool;
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  a.window_left = -1;
  a.num_qo_heads = p->num_qo_heads;
  a.group = p->num_qo_heads / p->num_kv_heads;
  a.cta_tile_q = p->cta_tile_q;
  a.bounded = 1;
  a.part_o = reinterpret_cast<float*>(base + w.o);
  a.part_ml = reinterpret_cast<float*>(base + w.ml);
  a.part_row = p->dev + set.o_row;
  a.tok_parts = p->dev + set.o_tok;
  a.beside = set.beside;
  if (set.beside > 0) a.part_clusters = std::max(1, (sm_count() - set.beside) / 2);
  a.status = status;
  wait_settings(&a.wait_ns, &a.test_withhold);
  return a;
}
cudaError_t shared_join(const pg_plan* p, const PartSet& set, pg_bf16_t* out, float* lse, unsigned char* base, const SharedWs& w,
                        cudaStream_t stream) {
  SharedJoinArgs j{};
  j.part_o = reinterpret_cast<const float*>(base + w.o);
  j.part_ml = reinterpret_cast<const float*>(base + w.ml);
  j.tok_parts = p->dev + set.o_tok;
  j.out = reinterpret_cast<__nv_bfloat16*>(out);
  j.own_lse = reinterpret_cast<const float*>(base + w.lse);
  j.lse = lse;
  j.num_tokens = p->num_tokens;
  j.num_qo_heads = p->num_qo_heads;
  return launch_shared_join(j, p->head_dim, stream);
}
// checks that both shared entries make before anything is launched
int check_shared(const pg_plan* plan, const pg_bf16_t* q, const pg_bf16_t* out, const float* lse, float sm_scale,
                 cudaStream_t stream) {
  int rc = check_bounded_plan(plan, stream);
  if (rc) return rc;
  if (!plan->own) return PG_ERR_PLAN_MISMATCH;
  if ((rc = check_bounded_attn(plan, 0))) return rc;
  // the rows of a group are counted on from the prefix's end
  if ((int64_t)plan->max_pos_end + plan->num_tokens > kLastEnd) return PG_ERR_I32_OVERFLOW;
  if (!fits_i32((int64_t)plan->num_tokens * plan->num_qo_heads)) return PG_ERR_I32_OVERFLOW;  // the join's grid
  if ((rc = check_attn_args(plan, plan->head_dim, -1, sm_scale))) return rc;
  if (plan->num_tokens == 0) return PG_OK;
  return check_attn_rows(q, out, lse);
}

int shared_attn(const pg_plan* plan, const pg_pool_t* pool, int32_t layer, const pg_bf16_t* q, pg_bf16_t* out,
                float* lse, float sm_scale, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_shared(plan, q, out, lse, sm_scale, stream);
  if (rc) return rc;
  const int32_t D = plan->head_dim;
  if ((rc = check_plan_pool(plan, pool, layer, D))) return rc;
  if ((int64_t)pool->num_pages * 2 * pool->num_kv_heads * pool->page_size > INT32_MAX)
    return PG_ERR_I32_OVERFLOW;  // tensor-map row coordinates are int32
  if (plan->num_tokens == 0) return PG_OK;
  const pg_plan* own = plan->own.get();
  SharedWs w;
  if (!shared_ws(plan, std::max(workspace_bytes(own), bounded_ws_bytes(own)), &w) || !ws ||
      ws_bytes < shared_workspace_bytes(plan))
    return PG_ERR_WORKSPACE;
  if (!aligned16(ws)) return PG_ERR_ALIGN;
  Bounded b;
  if (plan->parts[0].plain)
    return attn_common(plan, pool, layer, D, q, out, lse, -1, sm_scale, ws, ws_bytes, stream, &b);
  ws_bytes -= kSharedPad;
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  unsigned char* const base = shared_base(ws);
  const PartSet& set = plan->parts[0];
  AttnArgs a = part_args(plan, set, pool_dev(pool, layer), plan->dev + plan->o_pre_pages, plan->num_page_ids, q, sm_scale,
                         base, w, st);
  if (launch_attn_parts(a, D, stream) != cudaSuccess) return PG_ERR_CUDA;
  a.join_lse = lse;
  if (plan->decode) b.parts = &a;  // (the decode's join takes the parts along)
  rc = attn_common(own, pool, layer, D, q, out, reinterpret_cast<float*>(base + w.lse), -1, sm_scale, base + w.own,
                   ws_bytes - w.own, stream, &b);
  if (rc != PG_OK || b.parts) return rc;
  return shared_join(plan, set, out, lse, base, w, stream) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

// The 8-bit form: each prefix's pages are read back to the end of the workspace.
struct SharedQ8Ws {
  SharedWs w;
  size_t pages, page_bytes;
};
bool shared_q8_ws(const pg_plan* p, SharedQ8Ws* x) {
  const size_t own = q8_workspace_bytes(p->own.get());
  if (own > ((size_t)1 << 60) || !shared_ws(p, align256(own), &x->w)) return false;
  x->page_bytes = (size_t)4 * p->num_kv_heads * p->page_size * p->head_dim;
  x->pages = align1k(x->w.bytes);
  const __int128 end = (__int128)x->page_bytes * std::max(p->prefix_pages, 1) + x->pages;
  if (end > ((__int128)1 << 61)) return false;
  x->w.bytes = (size_t)end;
  return true;
}
size_t shared_q8_workspace_bytes(const pg_plan* p) {
  if (!p || !p->own || p->num_req == 0) return 0;
  SharedQ8Ws x;
  return shared_q8_ws(p, &x) ? std::max(x.w.bytes + kSharedPad, q8_workspace_bytes(p)) : SIZE_MAX;
}

int shared_q8_attn(const pg_plan* plan, const pg_q8_pool_t* pool, int32_t layer, const pg_bf16_t* q, pg_bf16_t* out,
                   float* lse, float sm_scale, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = check_shared(plan, q, out, lse, sm_scale, stream);
  if (rc) return rc;
  if ((rc = check_plan_q8(plan, pool, layer, 1))) return rc;
  const int32_t D = plan->head_dim, ps = plan->page_size, H = plan->num_kv_heads;
  if (plan->num_tokens == 0) return PG_OK;
  SharedQ8Ws x;
  if (!shared_q8_ws(plan, &x) || !ws || ws_bytes < shared_q8_workspace_bytes(plan)) return PG_ERR_WORKSPACE;
  if (!aligned16(ws)) return PG_ERR_ALIGN;
  if (plan->parts[1].plain)
    return q8_attn(plan, pool, layer, q, out, lse, -1, 0, sm_scale, ws, ws_bytes, stream);
  ws_bytes -= kSharedPad;
  unsigned char* const base = shared_base(ws);
  // a captured call's prefixes may come to hold as many pages as the workspace has room for
  const bool captured = capturing(stream);
  const int64_t room = captured ? (int64_t)((ws_bytes - x.pages) / x.page_bytes) : std::max(plan->prefix_pages, 1);
  const int32_t pages = (int32_t)std::min<int64_t>(room, plan->num_page_ids);
  if ((int64_t)std::max(pages, plan->num_page_ids) * 2 * H * ps > INT32_MAX) return PG_ERR_I32_OVERFLOW;
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  const PartSet& set = plan->parts[1];
  DequantArgs d{};
  d.plan = plan_dev(plan);
  d.plan.page_ids = plan->dev + plan->o_pre_pages;
  d.plan.num_page_ids = pages;
  d.src = q8_dev(pool, layer);
  d.dst = reinterpret_cast<__nv_bfloat16*>(base + x.pages);
  d.num_pages = pool->num_pages;
  d.page_size = ps;
  d.num_kv_heads = H;
  d.head_dim = D;
  d.num_layers = 1;
  d.list = 1;
  d.whole = plan->dev + set.o_live + 2;
  d.window_left = -1;
  d.status = st;
  if (launch_dequant(d, stream) != cudaSuccess) return PG_ERR_CUDA;
  PoolDev copy = q8_geometry(pool);
  copy.layer_base = d.dst;
  copy.num_pages = pages;
  AttnArgs a = part_args(plan, set, copy, nullptr, pages, q, sm_scale, base, x.w, st);
  if (launch_attn_parts(a, D, stream) != cudaSuccess) return PG_ERR_CUDA;
  a.join_lse = lse;
  const bool along = q8_direct(plan->own.get());  // the decode's join takes the parts along
  rc = q8_attn(plan->own.get(), pool, layer, q, out, reinterpret_cast<float*>(base + x.w.lse), -1, 0, sm_scale,
               base + x.w.own, x.pages - x.w.own, stream, along ? &a : nullptr);
  if (rc != PG_OK || along) return rc;
  return shared_join(plan, set, out, lse, base, x.w, stream) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

// Builds *plan (null) or updates it. No exception leaves a C entry: memory that the host cannot give is
// an argument that cannot be served, and nothing has changed by then.
template <class... Args>
int make_plan(pg_plan_t* plan, cudaStream_t stream, const Args&... args) {
  if (!plan) return PG_ERR_ARG;
  if (*plan && (*plan)->stream != stream) return PG_ERR_STREAM;
  pg_plan* p = *plan ? *plan : new (std::nothrow) pg_plan();
  if (!p) return PG_ERR_ARG;
  int rc = PG_ERR_ARG;
  try {
    rc = build_plan(p, args...);
  } catch (const std::exception&) {  // std::bad_alloc, std::length_error: before any CUDA call
  }
  if (rc != PG_OK && !*plan) {
    free_stage(&p->stage);
    delete p;
    return rc;
  }
  *plan = p;
  return rc;
}

// The device's status word if it already exists; never allocates.
int* status_word_existing(int* err) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) {
    *err = PG_ERR_CUDA;
    return nullptr;
  }
  std::lock_guard<std::mutex> lk(g_status_mu);
  *err = g_status_dev[dev] ? PG_OK : PG_ERR_CUDA;
  return g_status_dev[dev];
}

}  // namespace

extern "C" {

int pg_plan_paged_prefill(pg_plan_t* plan, int32_t num_req, const int64_t* qo_indptr,
                          const int64_t* kv_page_indptr, const int32_t* page_ids,
                          const int32_t* last_page_len, const int64_t* start_pos,
                          int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                          int32_t page_size, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return make_plan(plan, s, num_req, qo_indptr, kv_page_indptr, page_ids, last_page_len, start_pos,
                   num_qo_heads, num_kv_heads, head_dim, page_size, s);
}

int pg_plan_paged_prefill_ring(pg_plan_t* plan, int32_t num_req, const int64_t* qo_indptr,
                               const int64_t* kv_page_indptr, const int32_t* page_ids,
                               const int64_t* start_pos, int32_t num_qo_heads,
                               int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               int32_t window_left, pg_stream_t stream) {
  if (!plan) return PG_ERR_ARG;
  if (window_left < 0) return PG_ERR_WINDOW;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return make_plan(plan, s, num_req, qo_indptr, kv_page_indptr, page_ids, nullptr, start_pos,
                   num_qo_heads, num_kv_heads, head_dim, page_size, s, window_left);
}

int pg_plan_paged_segment(pg_plan_t* plan, int32_t num_req, const int64_t* qo_indptr,
                          const int64_t* kv_page_indptr, const int32_t* page_ids,
                          const int32_t* last_page_len, const int64_t* kv_start,
                          const int64_t* start_pos, int32_t num_qo_heads, int32_t num_kv_heads,
                          int32_t head_dim, int32_t page_size, pg_stream_t stream) {
  if (!plan) return PG_ERR_ARG;
  if (num_req > 0 && !kv_start) return PG_ERR_ARG;
  static const int64_t kNoSegments = 0;  // a non-null pointer for an empty batch
  const int64_t* ks = kv_start ? kv_start : &kNoSegments;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return make_plan(plan, s, num_req, qo_indptr, kv_page_indptr, page_ids, last_page_len, start_pos,
                   num_qo_heads, num_kv_heads, head_dim, page_size, s, -1, ks);
}

int pg_plan_paged_shared(pg_plan_t* plan, int32_t num_req, const int64_t* qo_indptr,
                         const int64_t* kv_page_indptr, const int32_t* page_ids,
                         const int32_t* last_page_len, const int64_t* start_pos, int32_t num_groups,
                         const int64_t* group_indptr, const int64_t* prefix_len, int32_t num_qo_heads,
                         int32_t num_kv_heads, int32_t head_dim, int32_t page_size, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Groups g;
  g.num = num_groups;
  g.indptr = group_indptr;
  g.prefix = prefix_len;
  return make_plan(plan, s, num_req, qo_indptr, kv_page_indptr, page_ids, last_page_len, start_pos,
                   num_qo_heads, num_kv_heads, head_dim, page_size, s, -1, nullptr, &g);
}

void pg_plan_destroy(pg_plan_t plan) {
  if (!plan) return;
  if (plan->dev) cudaFreeAsync(plan->dev, plan->stream);
  free_stage(&plan->stage);
  delete plan;
}

int pg_plan_info(const pg_plan_t p, pg_plan_info_t* info) {
  if (!p || !info) return PG_ERR_ARG;
  info->num_req = p->num_req; info->num_tokens = p->num_tokens;
  info->num_qo_heads = p->num_qo_heads; info->num_kv_heads = p->num_kv_heads;
  info->head_dim = p->head_dim; info->page_size = p->page_size;
  info->max_page_id = p->max_page_id; info->max_last_page_len = p->max_last_page_len;
  info->max_qo_len = p->max_qo_len; info->max_kv_len = p->max_kv_len;
  info->max_pos_end = p->max_pos_end; info->cta_tile_q = p->cta_tile_q;
  info->decode = p->decode; info->kv_chunk = p->kv_chunk; info->max_chunks = p->max_chunks;
  info->num_work = p->num_work;
  info->d_page_ids = p->dev + p->o_pages;
  info->stream = reinterpret_cast<pg_stream_t>(p->stream);
  info->metadata_bytes = (int64_t)p->dev_elems * (int64_t)sizeof(int32_t);
  return PG_OK;
}

int pg_rope_table(float* rope_cos, float* rope_sin, int32_t rows, int32_t head_dim, double theta,
                  pg_stream_t stream) {
  if (!rope_cos || !rope_sin || rows < 1 || head_dim < 2 || head_dim % 2) return PG_ERR_ARG;
  if (!std::isfinite(theta) || !(theta > 0.0)) return PG_ERR_NONFINITE;
  int64_t n = 0;
  if (!mul_i64(rows, head_dim / 2, &n) || !fits_i32(n)) return PG_ERR_I32_OVERFLOW;
  cudaError_t e = launch_rope_table(rope_cos, rope_sin, rows, head_dim, theta,
                                    reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_prep_paged_hd256(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                        const pg_bf16_t* q_raw, int64_t q_tok_stride, const pg_bf16_t* k_raw,
                        int64_t k_tok_stride, const pg_bf16_t* v_raw, int64_t v_tok_stride,
                        const pg_bf16_t* w_q, const pg_bf16_t* w_k, float eps,
                        const float* rope_cos, const float* rope_sin, int32_t rope_rows,
                        pg_bf16_t* q_out, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PrepArgs a;
  int rc = prep_common(plan, PrepPool{pool, nullptr}, layer, 256, q_raw, q_tok_stride, k_raw, k_tok_stride, v_raw,
                       v_tok_stride, w_q, w_k, eps, rope_cos, rope_sin, rope_rows, q_out, s, &a);
  if (rc != PG_OK || plan->num_tokens == 0) return rc;
  return launch_prep_hd256(a, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_prep_paged_hd512(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                        const pg_bf16_t* q_raw, int64_t q_tok_stride, const pg_bf16_t* k_raw,
                        int64_t k_tok_stride, const pg_bf16_t* w_q, const pg_bf16_t* w_k,
                        float eps, const float* rope_cos, const float* rope_sin,
                        int32_t rope_rows, pg_bf16_t* q_out, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PrepArgs a;
  int rc = prep_common(plan, PrepPool{pool, nullptr}, layer, 512, q_raw, q_tok_stride, k_raw, k_tok_stride, nullptr,
                       0, w_q, w_k, eps, rope_cos, rope_sin, rope_rows, q_out, s, &a);
  if (rc != PG_OK || plan->num_tokens == 0) return rc;
  return launch_prep_hd512(a, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

size_t pg_workspace_bytes(const pg_plan_t plan) {
  return workspace_bytes(plan);
}

int pg_attn_paged_prefill(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                          const pg_bf16_t* q, pg_bf16_t* out, int32_t window_left, float sm_scale,
                          void* workspace, size_t ws_bytes, pg_stream_t stream) {
  return attn_common(plan, pool, layer, 256, q, out, nullptr, window_left, sm_scale, workspace, ws_bytes,
                     reinterpret_cast<cudaStream_t>(stream));
}

int pg_attn_paged_prefill_hd512(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                                const pg_bf16_t* q, pg_bf16_t* out, int32_t window_left,
                                float sm_scale, void* workspace, size_t ws_bytes,
                                pg_stream_t stream) {
  return attn_common(plan, pool, layer, 512, q, out, nullptr, window_left, sm_scale, workspace, ws_bytes,
                     reinterpret_cast<cudaStream_t>(stream));
}

int pg_attn_paged_prefill_lse(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                              const pg_bf16_t* q, pg_bf16_t* out, float* lse,
                              int32_t window_left, float sm_scale, void* workspace,
                              size_t ws_bytes, pg_stream_t stream) {
  if (!lse && plan && plan->num_tokens > 0) return PG_ERR_ARG;
  return attn_common(plan, pool, layer, 256, q, out, lse, window_left, sm_scale, workspace,
                     ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int pg_attn_paged_prefill_hd512_lse(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                                    const pg_bf16_t* q, pg_bf16_t* out, float* lse,
                                    int32_t window_left, float sm_scale, void* workspace,
                                    size_t ws_bytes, pg_stream_t stream) {
  if (!lse && plan && plan->num_tokens > 0) return PG_ERR_ARG;
  return attn_common(plan, pool, layer, 512, q, out, lse, window_left, sm_scale, workspace,
                     ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

int pg_merge_attn_states(const pg_bf16_t* out_a, const float* lse_a, const pg_bf16_t* out_b,
                         const float* lse_b, pg_bf16_t* out, float* lse, int64_t rows,
                         int32_t head_dim, pg_stream_t stream) {
  if (rows < 0 || head_dim <= 0 || head_dim % 8 != 0) return PG_ERR_ARG;
  if (rows > INT32_MAX) return PG_ERR_I32_OVERFLOW;
  if (rows == 0) return PG_OK;
  if (!out_a || !lse_a || !out_b || !lse_b || !out) return PG_ERR_ARG;
  if (!aligned16(out_a) || !aligned16(out_b) || !aligned16(out)) return PG_ERR_ALIGN;
  if (((uintptr_t)lse_a & 3u) || ((uintptr_t)lse_b & 3u) || ((uintptr_t)lse & 3u))
    return PG_ERR_ALIGN;
  const cudaError_t e = launch_merge_states(
      reinterpret_cast<const __nv_bfloat16*>(out_a), lse_a,
      reinterpret_cast<const __nv_bfloat16*>(out_b), lse_b,
      reinterpret_cast<__nv_bfloat16*>(out), lse, (int32_t)rows, head_dim,
      reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_attn_paged_sink(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                       const pg_bf16_t* q, pg_bf16_t* out, float* lse, int32_t window_left,
                       int32_t num_sink, float sm_scale, void* workspace, size_t ws_bytes,
                       pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = check_bounded_plan(plan, s);
  if (rc || (rc = check_bounded_attn(plan, num_sink))) return rc;
  Bounded b;
  b.num_sink = num_sink;
  return attn_common(plan, pool, layer, plan->head_dim, q, out, lse, window_left, sm_scale, workspace,
                     ws_bytes, s, &b);
}

size_t pg_sink_workspace_bytes(const pg_plan_t plan) {
  return std::max(workspace_bytes(plan), bounded_ws_bytes(plan));
}

size_t pg_mass_workspace_bytes(const pg_plan_t plan) { return mass_workspace_bytes(plan); }

int pg_attn_paged_mass(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                       const pg_bf16_t* q, pg_bf16_t* out, float* lse, const pg_kv_stats_t* stats,
                       int32_t window_left, int32_t num_sink, float sm_scale, void* workspace,
                       size_t ws_bytes, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = check_bounded_plan(plan, s);
  if (rc || (rc = check_bounded_attn(plan, num_sink))) return rc;
  if ((rc = check_plan_pool(plan, pool, layer, plan->head_dim))) return rc;
  if ((rc = check_stats(plan, stats, layer, 1))) return rc;
  if (stats->num_layers != pool->num_layers || stats->num_pages != pool->num_pages)
    return PG_ERR_LAYOUT;
  bool shared = false;
  if ((rc = shares_pages(plan, &shared))) return rc;
  if (shared) return PG_ERR_SHARED_PAGE;
  if (plan->num_tokens > 0 && !lse) return PG_ERR_ARG;
  const size_t need = mass_workspace_bytes(plan);
  if (need > 0) {
    if (!workspace || ws_bytes < need) return PG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PG_ERR_ALIGN;
  }
  // every grid fits: at most a block per 64 keys of a head, and (decode) one per 128 output columns
  int64_t blocks = 0, joins = 0;
  if (!mul_i64((plan->max_seen + 63) / 64, plan->num_req, &blocks) ||
      !mul_i64(blocks, plan->num_kv_heads, &blocks) ||
      !mul_i64((int64_t)plan->num_req * plan->num_qo_heads, plan->head_dim / 64, &joins) ||
      !fits_i32(blocks + joins))
    return PG_ERR_I32_OVERFLOW;
  Bounded b;
  b.num_sink = num_sink;
  b.stats = stats_dev(stats, layer);
  const size_t attn_ws = align256(bounded_ws_bytes(plan));
  if (plan->decode && plan->num_req > 0) {
    b.logits = reinterpret_cast<float*>(static_cast<char*>(workspace) + attn_ws);
    // as many as the workspace holds: a graph's plan may grow into a larger one
    b.logit_slots = (int64_t)((ws_bytes - attn_ws) / ((size_t)plan->num_qo_heads * sizeof(float)));
  }
  MassArgs m{};
  rc = attn_common(plan, pool, layer, plan->head_dim, q, out, lse, window_left, sm_scale, workspace,
                   attn_ws, s, &b, &m.attn);
  if (rc != PG_OK || plan->num_tokens == 0) return rc;
  m.ws = workspace;  // (prefill attention itself needs none)
  // (the tensor-core decode adds the weights itself)
  const bool done = plan->decode && bounded_tc(plan);
  const cudaError_t e = done           ? cudaSuccess
                        : plan->decode ? launch_mass_decode(m, s)
                                       : launch_mass_prefill(m, plan->head_dim, s);
  return e == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_prep_paged_q8(const pg_plan_t plan, const pg_q8_pool_t* pool, int32_t layer, const pg_bf16_t* q_raw,
                     int64_t q_tok_stride, const pg_bf16_t* k_raw, int64_t k_tok_stride, const pg_bf16_t* v_raw,
                     int64_t v_tok_stride, const pg_bf16_t* w_q, const pg_bf16_t* w_k, float eps,
                     const float* rope_cos, const float* rope_sin, int32_t rope_rows, pg_bf16_t* q_out,
                     pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = check_bounded_plan(plan, s);
  if (rc) return rc;
  if (!pool) return PG_ERR_ARG;
  if (plan->head_dim == 512 && v_raw) return PG_ERR_ARG;  // V is the norm of the raw K
  PrepArgs a;
  rc = prep_common(plan, PrepPool{nullptr, pool}, layer, plan->head_dim, q_raw, q_tok_stride, k_raw, k_tok_stride,
                   v_raw, plan->head_dim == 512 ? 0 : v_tok_stride, w_q, w_k, eps, rope_cos, rope_sin, rope_rows,
                   q_out, s, &a);
  if (rc != PG_OK || plan->num_tokens == 0) return rc;
  return launch_prep_q8(a, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_kv_dequantize(const pg_plan_t plan, const pg_q8_pool_t* src, const pg_pool_t* dst, int32_t layer,
                     int32_t num_layers, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = check_bounded_plan(plan, s);
  if (rc || (rc = check_plan_q8(plan, src, layer, num_layers))) return rc;
  if ((rc = check_plan_pool(plan, dst, layer, plan->head_dim))) return rc;
  if (layer > dst->num_layers - num_layers) return PG_ERR_LAYER;
  int64_t tasks = 0;
  if (!mul_i64((int64_t)num_layers * plan->num_page_ids, (int64_t)2 * plan->num_kv_heads, &tasks) || !fits_i32(tasks))
    return PG_ERR_I32_OVERFLOW;
  if (plan->num_req == 0) return PG_OK;
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  DequantArgs d{};
  d.plan = plan_dev(plan);
  d.src = q8_dev(src, layer);
  d.dst = pool_dev(dst, layer).layer_base;
  d.dst_stride_layer = dst->stride_layer;
  d.num_pages = std::min(src->num_pages, dst->num_pages);
  d.page_size = plan->page_size;
  d.num_kv_heads = plan->num_kv_heads;
  d.head_dim = plan->head_dim;
  d.num_layers = num_layers;
  d.window_left = -1;
  d.status = st;
  return launch_dequant(d, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

size_t pg_q8_workspace_bytes(const pg_plan_t plan) { return q8_workspace_bytes(plan); }

int pg_attn_paged_q8(const pg_plan_t plan, const pg_q8_pool_t* pool, int32_t layer, const pg_bf16_t* q, pg_bf16_t* out,
                     float* lse, int32_t window_left, int32_t num_sink, float sm_scale, void* workspace,
                     size_t ws_bytes, pg_stream_t stream) {
  return q8_attn(plan, pool, layer, q, out, lse, window_left, num_sink, sm_scale, workspace, ws_bytes,
                 reinterpret_cast<cudaStream_t>(stream));
}

size_t pg_shared_workspace_bytes(const pg_plan_t plan) { return shared_workspace_bytes(plan); }

int pg_attn_paged_shared(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer, const pg_bf16_t* q, pg_bf16_t* out,
                         float* lse, float sm_scale, void* workspace, size_t ws_bytes, pg_stream_t stream) {
  return shared_attn(plan, pool, layer, q, out, lse, sm_scale, workspace, ws_bytes,
                     reinterpret_cast<cudaStream_t>(stream));
}

size_t pg_shared_q8_workspace_bytes(const pg_plan_t plan) { return shared_q8_workspace_bytes(plan); }

int pg_attn_paged_shared_q8(const pg_plan_t plan, const pg_q8_pool_t* pool, int32_t layer, const pg_bf16_t* q,
                            pg_bf16_t* out, float* lse, float sm_scale, void* workspace, size_t ws_bytes,
                            pg_stream_t stream) {
  return shared_q8_attn(plan, pool, layer, q, out, lse, sm_scale, workspace, ws_bytes,
                        reinterpret_cast<cudaStream_t>(stream));
}

int pg_kv_evict_select(const pg_plan_t plan, const pg_kv_stats_t* stats, int32_t layer,
                       int32_t num_layers, int32_t budget, int32_t num_sink, int32_t num_recent,
                       int32_t* src, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  EvictArgs a;
  if (num_sink < 0 || num_recent < 0 || (int64_t)num_sink + num_recent > budget) return PG_ERR_ARG;
  const int rc = evict_common(plan, stats, layer, num_layers, budget, src, s, &a);
  if (rc != PG_OK || plan->num_req == 0) return rc;
  a.num_sink = num_sink;
  a.num_recent = num_recent;
  return launch_evict_select(a, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_kv_evict_apply(const pg_plan_t plan, const pg_pool_t* pool, const pg_kv_stats_t* stats,
                      int32_t layer, int32_t num_layers, int32_t budget, const int32_t* src,
                      pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  EvictArgs a;
  int rc = evict_common(plan, stats, layer, num_layers, budget, src, s, &a);
  if (rc) return rc;
  if ((rc = check_plan_pool(plan, pool, layer, plan->head_dim))) return rc;
  if (stats->num_layers != pool->num_layers || stats->num_pages != pool->num_pages)
    return PG_ERR_LAYOUT;
  if (plan->head_dim != 256 && plan->head_dim != 512) return PG_ERR_PLAN_MISMATCH;
  if (plan->num_req == 0) return PG_OK;
  a.pool = pool_dev(pool, layer);
  a.pool_stride_layer = pool->stride_layer;
  return launch_evict_apply(a, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_attn_paged_decode_noalloc(const pg_plan_t plan, const pg_pool_t* pool, int32_t layer,
                                 const pg_bf16_t* q, pg_bf16_t* out, int32_t window_left,
                                 float sm_scale, pg_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!plan) return PG_ERR_ARG;
  if (s != plan->stream) return PG_ERR_STREAM;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PG_ERR_CUDA;
  if (dev != plan->device) return PG_ERR_STREAM;
  if (!plan->decode && plan->num_req > 0) return PG_ERR_PLAN_MISMATCH;
  if (workspace_bytes(plan) > PG_NOALLOC_SCRATCH_BYTES) return PG_ERR_WORKSPACE;
  const int32_t D = plan->head_dim;
  if (D != 256 && D != 512) return PG_ERR_PLAN_MISMATCH;
  int rc = check_plan_pool(plan, pool, layer, D);
  if (rc) return rc;
  const int32_t group = plan->num_qo_heads / plan->num_kv_heads;
  const int32_t kernel_cta = attn_kernel_cta_tile_q(D, group, plan->page_size);
  if (kernel_cta == 0 || kernel_cta != plan->cta_tile_q) return PG_ERR_PLAN_MISMATCH;
  if (attn_kernel_kv_chunk(D) != plan->kv_chunk) return PG_ERR_PLAN_MISMATCH;
  if (window_left < -1) return PG_ERR_WINDOW;
  if (plan->ring && (window_left < 0 || window_left > plan->ring_window)) return PG_ERR_WINDOW;
  if (!std::isfinite(sm_scale)) return PG_ERR_NONFINITE;
  if (attn_decode_stream_supported(D, group, plan->page_size) &&
      (int64_t)pool->num_pages * 2 * pool->num_kv_heads * pool->page_size > INT32_MAX)
    return PG_ERR_I32_OVERFLOW;  // tensor-map row coordinates are int32
  if (!attn_decode_stream_supported(D, group, plan->page_size) && plan->max_chunks > 65535)
    return PG_ERR_I32_OVERFLOW;  // the chunked kernel's grid z dimension
  if (plan->num_tokens == 0) return PG_OK;
  if (!q || !out) return PG_ERR_ARG;
  if (!aligned16(q) || !aligned16(out)) return PG_ERR_ALIGN;
  int err = PG_OK;
  int* st = status_word_existing(&err);
  if (!st) return err;
  AttnArgs a{};
  a.plan = plan_dev(plan);
  a.pool = pool_dev(pool, layer);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = nullptr;
  a.ws_raw = nullptr;
  a.ws_o = nullptr;
  a.ws_ml = nullptr;
  a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  a.window_left = window_left;
  a.num_qo_heads = plan->num_qo_heads;
  a.group = group;
  a.cta_tile_q = plan->cta_tile_q;
  a.kv_chunk = plan->kv_chunk;
  a.max_chunks = plan->max_chunks;
  a.status = st;
  wait_settings(&a.wait_ns, &a.test_withhold);
  return launch_attn_decode_static(a, D, s) == cudaSuccess ? PG_OK : PG_ERR_CUDA;
}

int pg_device_status(pg_stream_t stream) {
  int err = PG_OK;
  int* st = status_word(&err);
  if (!st) return err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int h = 0;
  if (cudaMemcpyAsync(&h, st, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return PG_ERR_CUDA;
  if (cudaMemsetAsync(st, 0, sizeof(int), s) != cudaSuccess) return PG_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return PG_ERR_CUDA;
  if (h & kStatusTimeout) return PG_ERR_DEVICE_TIMEOUT;
  return h ? PG_ERR_DEVICE_BOUNDS : PG_OK;
}

int64_t pg_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int pg_test_shared_form(int32_t form) {
  if (form < 0 || form > 2) return PG_ERR_ARG;
  g_test_shared.store(form, std::memory_order_relaxed);
  return PG_OK;
}

int pg_test_bounded_wait(int32_t withhold, int64_t wait_limit_ns) {
  if (withhold == 0) {
    g_test_withhold.store(0, std::memory_order_relaxed);
    g_wait_ns.store(kDefaultWaitNs, std::memory_order_relaxed);
    return PG_OK;
  }
  if (withhold != 1 || wait_limit_ns < 1000000 || wait_limit_ns > (int64_t)kDefaultWaitNs)
    return PG_ERR_ARG;
  g_wait_ns.store((uint64_t)wait_limit_ns, std::memory_order_relaxed);
  g_test_withhold.store(1, std::memory_order_relaxed);
  return PG_OK;
}

const char* pg_status_string(int s) {
  switch (s) {
    case PG_OK: return "ok";
    case PG_ERR_ARG: return "invalid argument (null pointer, negative count, bad indptr)";
    case PG_ERR_PAGE_OOB: return "page id outside the pool";
    case PG_ERR_LAST_PAGE_LEN: return "last_page_len outside [1, page_size]";
    case PG_ERR_I32_OVERFLOW: return "length or offset does not fit int32 (or stride product int64)";
    case PG_ERR_ZERO_KV_HEADS: return "num_kv_heads is zero";
    case PG_ERR_HEADS: return "num_qo_heads is not a positive multiple of num_kv_heads";
    case PG_ERR_NONFINITE: return "non-finite or non-positive scale, eps or theta";
    case PG_ERR_ROPE_RANGE: return "a position is past the rotary tables";
    case PG_ERR_COVERAGE: return "pages do not cover the keys the step needs (linear: exactly [0, start_pos + qo_len))";
    case PG_ERR_LAYER: return "layer outside the pool";
    case PG_ERR_LAYOUT: return "pool layout, strides or capacity inconsistent";
    case PG_ERR_PLAN_MISMATCH: return "plan geometry or tiling disagrees with the pool or kernel";
    case PG_ERR_WINDOW: return "window_left below -1";
    case PG_ERR_WORKSPACE: return "workspace missing or too small";
    case PG_ERR_STREAM: return "stream differs from the plan's stream";
    case PG_ERR_CUDA: return "CUDA runtime error";
    case PG_ERR_DEVICE_BOUNDS: return "a kernel skipped an out-of-range access";
    case PG_ERR_ALIGN: return "pointer or stride not 16-byte aligned";
    case PG_ERR_SHARED_PAGE: return "a page is listed twice where each needs its own";
    case PG_ERR_DEVICE_TIMEOUT: return "a kernel gave up a bounded wait and returned early";
    default: return "unknown status";
  }
}

}  // extern "C"
