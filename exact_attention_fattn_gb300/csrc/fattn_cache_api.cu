// C-ABI boundary of the paged 8-bit cache: argument checks, tensor maps,
// workspace layout and the choice of kernel.  See include/fattn.h.
#include <math.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/fattn.h"
#include "fattn_internal.h"

namespace fattn {
namespace {

struct NvtxScope {
  explicit NvtxScope(const char* name) { nvtxRangePushA(name); }
  ~NvtxScope() { nvtxRangePop(); }
  NvtxScope(const NvtxScope&) = delete;
  NvtxScope& operator=(const NvtxScope&) = delete;
};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kMaxSeqs = 4096;
constexpr int kMaxKvHeads = 1024;
constexpr int kMaxGroup = 128;

int check_cache(const fattn_cache* c) {
  if (!c) return FATTN_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FATTN_ERR_UNSUPPORTED;
  if (c->page != 32 && c->page != 64 && c->page != 128) return FATTN_ERR_UNSUPPORTED;
  if (c->pages <= 0 || c->Hkv <= 0 || c->Hkv > kMaxKvHeads) return FATTN_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return FATTN_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || !aligned(c->k_bounds, 16))
    return FATTN_ERR_INVALID_ARG;
  const long long least = static_cast<long long>(c->Hkv) * c->page * c->d;
  if (c->page_stride < least || c->page_stride % 16 != 0 || c->page_stride >= (1ll << 40))
    return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int check_batch(const fattn_cache* c, const int* page_table, const int* q_start, const int* kv_len,
                int T, int B, int max_pages) {
  if (!page_table || !q_start || !kv_len) return FATTN_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4))
    return FATTN_ERR_INVALID_ARG;
  if (T <= 0 || B <= 0 || B > kMaxSeqs || max_pages <= 0) return FATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * c->page > 0x7fff0000ll) return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int check_heads(const fattn_cache* c, int T, int Hq) {
  if (Hq <= 0 || Hq % c->Hkv != 0 || Hq / c->Hkv > kMaxGroup) return FATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * Hq > 0x7fffffffll) return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int check_rows(const void* p, long long row, long long least) {
  if (!p || !aligned(p, 16) || row < least || row % 8 != 0) return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int page_shift(int page) { return page == 32 ? 5 : (page == 64 ? 6 : 7); }

CacheSeqs seqs_of(const int* page_table, const int* q_start, const int* kv_len, int T, int B,
                  int max_pages) {
  CacheSeqs s;
  s.q_start = q_start;
  s.kv_len = kv_len;
  s.table = page_table;
  s.T = T;
  s.B = B;
  s.max_pages = max_pages;
  return s;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Partial results of the units that CTAs share, two per CTA, and, for the
// tcgen05 kernel, the call's q_rows queries in two parts.
struct AttnWorkspace {
  size_t o_off, ml_off, rec_off, q_off, qs_off, total;
};

AttnWorkspace attn_workspace(int rows, int d, size_t q_rows) {
  AttnWorkspace w;
  const size_t slots = static_cast<size_t>(part_rows(d, rows));
  w.o_off = 0;
  w.ml_off = align256(slots * d * sizeof(float));
  w.rec_off = w.ml_off + align256(slots * sizeof(float2));
  w.q_off = w.rec_off + align256(slots / rows * sizeof(int4));
  if (rows != kChunkRows) q_rows = 0;
  w.qs_off = w.q_off + 2 * align256(q_rows * d);
  w.total = w.qs_off + align256(q_rows * sizeof(float));
  return w;
}

// Which kernel: units of 16 rows on mma.sync, or of 256 on tcgen05.  Pages
// selected per token leave a unit the group's rows of one token.  Otherwise the rows of
// an average sequence decide: up to 16 are one unit; with 2 to 4 units a
// sequence the first kernel reads every key that often (out of L2 after the first
// time) but starts and ends sooner, so it takes small calls.  Measured, 8 kv
// heads, mma.sync / tcgen05 us: d = 128: 16 rows, 32 x 1000 tokens 29 / 45, 16 x
// 16000 93 / 128; 24 rows, 32 x 2000 57 / 59, 32 x 4000 94 / 84; 40 rows, 32 x 500
// 37 / 35, 32 x up to 4000 93 / 67; 64 rows, 8 x 1000 26.7 / 26.2, 1 x 8000 23.5 / 32,
// 32 x 500 46 / 36.  d = 64: 24 rows, 16 x 16000 103 / 123; 40 rows, 32 x 1000 36 /
// 42, 32 x 4000 86 / 80; 64 rows, 4 x 8000 37 / 33.
// tokens: at most as many times a kv head the call can reach, -1 for unknown.  The
// lengths are on the device, so this is what the page tables and the pool could
// hold; the measurements above are with tables as wide as the longest sequence.
// Where both are much larger than what is in use, 2 to 4 units go to tcgen05 however
// short the sequences are (exact table / table of 2048 pages and 16 times the pool,
// us: 64 rows, 1 x 8000 23.5 / 30.7, 8 x 1000 26.7 / 23.3; d = 64: 40 rows, 32 x 1000
// 31.4 / 37.3, 24 rows, 16 x 16000 82 / 98.5).  Likewise a batch that mixes pieces of
// prompts with single tokens is served as its average: 255 single tokens on 1000 to
// 4000 keys and a piece of 700 on 16000 take 962 us in one call, 212 + 153 in two.
bool few_rows(int T, int B, int group, int d, int n_selected, long long tokens) {
  const long long units = (static_cast<long long>(T) * group + kDecodeRows * static_cast<long long>(B) - 1) /
                          (kDecodeRows * static_cast<long long>(B));
  if (n_selected > 0 || units <= 1) return true;
  if (units > 4 || tokens < 0) return false;
  const long long limit = (units == 2 ? 1ll << 19 : 1ll << 16) * (d == 64 && units < 4 ? 4 : 1);
  return tokens <= limit;
}

}  // namespace

}  // namespace fattn

using namespace fattn;

extern "C" {

int fattn_cache_append(const fattn_cache* cache, const void* k_new, long long k_row,
                       const void* v_new, long long v_row, const void* q, long long q_row,
                       void* q_out, int Hq, const float* rope, int rope_len, int rope_dim,
                       int interleaved, const int* page_table, const int* q_start,
                       const int* kv_len, int T, int B, int max_pages, fattn_stream_t stream) {
  const NvtxScope nvtx_range("fattn_cache_append");
  int rc = check_cache(cache);
  if (rc != FATTN_OK) return rc;
  if ((rc = check_batch(cache, page_table, q_start, kv_len, T, B, max_pages)) != FATTN_OK) return rc;
  const long long kv_least = static_cast<long long>(cache->Hkv) * cache->d;
  if ((rc = check_rows(k_new, k_row, kv_least)) != FATTN_OK) return rc;
  if ((rc = check_rows(v_new, v_row, kv_least)) != FATTN_OK) return rc;
  if ((q == nullptr) != (q_out == nullptr)) return FATTN_ERR_INVALID_ARG;
  if (q) {
    if ((rc = check_heads(cache, T, Hq)) != FATTN_OK) return rc;
    const long long q_least = static_cast<long long>(Hq) * cache->d;
    if ((rc = check_rows(q, q_row, q_least)) != FATTN_OK) return rc;
    if (!aligned(q_out, 16) || (q_out == q && q_row != q_least)) return FATTN_ERR_INVALID_ARG;
  }
  if (rope) {
    if (!aligned(rope, 16) || rope_len <= 0 || rope_dim <= 0 || rope_dim > cache->d ||
        rope_dim % 16 != 0)
      return FATTN_ERR_INVALID_ARG;
  } else if (rope_dim != 0) {
    return FATTN_ERR_INVALID_ARG;
  }
  // one block per page and head at most, one per 8 groups of 8 heads of q, and one that checks the batch
  const long long blocks = (T / cache->page + 2ll * B) * cache->Hkv +
                           (q ? static_cast<long long>(T) * ((Hq + 7) / 8) / 8 + 1 : 0) + 1;
  if (blocks > 0x7fffffffll) return FATTN_ERR_INVALID_ARG;
  CacheAppendArgs a{};
  long long budget = 0;
  if ((rc = call_setup(&a.status, &budget)) != FATTN_OK) return rc;
  a.s = seqs_of(page_table, q_start, kv_len, T, B, max_pages);
  a.k = static_cast<uint8_t*>(cache->k);
  a.v = static_cast<uint8_t*>(cache->v);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.bounds = static_cast<int8_t*>(cache->k_bounds);
  a.page_stride = cache->page_stride;
  a.pages = cache->pages;
  a.Hkv = cache->Hkv;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_row = k_row;
  a.v_row = v_row;
  a.q_row = q_row;
  a.Hq = q ? Hq : 0;
  a.rope = rope;
  a.rope_len = rope_len;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved != 0;
  return launch_cache_append(cache->page, cache->d, a, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FATTN_OK
             : FATTN_ERR_CUDA;
}

size_t fattn_cache_fwd_workspace_bytes(int T, int B, int Hq, int Hkv, int d, int n_selected) {
  if (T <= 0 || B <= 0 || B > kMaxSeqs || Hkv <= 0 || Hkv > kMaxKvHeads || Hq <= 0 ||
      Hq % Hkv != 0 || Hq / Hkv > kMaxGroup || (d != 64 && d != 128) || n_selected < 0)
    return 0;
  // of the larger layout, where the cache's size decides
  return attn_workspace(few_rows(T, B, Hq / Hkv, d, n_selected, -1) ? kDecodeRows : kChunkRows, d,
                        static_cast<size_t>(T) * Hq)
      .total;
}

int fattn_cache_fwd(const fattn_cache* cache, const void* q, long long q_row, void* o, float* lse,
                    const int* page_table, const int* q_start, const int* kv_len,
                    const int* selected, int n_selected, void* workspace, size_t workspace_bytes,
                    int T, int B, int Hq, int max_pages, int causal, float scale,
                    fattn_stream_t stream) {
  const NvtxScope nvtx_range("fattn_cache_fwd");
  int rc = check_cache(cache);
  if (rc != FATTN_OK) return rc;
  if ((rc = check_batch(cache, page_table, q_start, kv_len, T, B, max_pages)) != FATTN_OK) return rc;
  if ((rc = check_heads(cache, T, Hq)) != FATTN_OK) return rc;
  if ((rc = check_rows(q, q_row, static_cast<long long>(Hq) * cache->d)) != FATTN_OK) return rc;
  if (!o || !aligned(o, 16) || !lse || !aligned(lse, 4)) return FATTN_ERR_INVALID_ARG;
  if ((selected == nullptr) != (n_selected == 0) || n_selected < 0 || !aligned(selected, 4))
    return FATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(n_selected) * cache->page > 0x7fff0000ll) return FATTN_ERR_INVALID_ARG;
  if (!isfinite(scale) || !(scale > 0.f)) return FATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < fattn_cache_fwd_workspace_bytes(T, B, Hq, cache->Hkv, cache->d, n_selected))
    return FATTN_ERR_INVALID_ARG;
  CacheAttnArgs a{};
  if ((rc = call_setup(&a.status, &a.wait_budget)) != FATTN_OK) return rc;
  a.s = seqs_of(page_table, q_start, kv_len, T, B, max_pages);
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.selected = selected;
  a.n_selected = n_selected;
  a.pages = cache->pages;
  a.Hkv = cache->Hkv;
  a.group = Hq / cache->Hkv;
  a.page_shift = page_shift(cache->page);
  a.causal = causal != 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  const long long reach = static_cast<long long>(B) * max_pages;
  const long long tokens = (reach < cache->pages ? reach : cache->pages) * cache->page * cache->Hkv;
  const bool few = few_rows(T, B, a.group, cache->d, n_selected, tokens);
  const int unit_rows = few ? kDecodeRows : kChunkRows, piece_keys = few ? kDecodeKeys : kChunkTileKeys;
  const size_t q_rows = static_cast<size_t>(T) * Hq;
  const AttnWorkspace w = attn_workspace(unit_rows, cache->d, q_rows);
  char* base = static_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(base + w.o_off);
  a.part_ml = reinterpret_cast<float2*>(base + w.ml_off);
  a.rec = reinterpret_cast<int4*>(base + w.rec_off);
  a.q_codes = reinterpret_cast<uint8_t*>(base + w.q_off);
  a.q_lo = static_cast<long long>(align256(q_rows * cache->d));
  a.q_scale = reinterpret_cast<float*>(base + w.qs_off);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FATTN_ERR_CUDA;
  const int max_ctas = (sms < kSms ? sms : kSms) * (few ? decode_ctas(cache->d) : kChunkCtas);
  // Pieces of keys of all units, at most (the lengths are on the device).
  const long long keys = static_cast<long long>(selected ? n_selected : max_pages) * cache->page;
  const long long units =
      (selected ? static_cast<long long>(T) * ((a.group + unit_rows - 1) / unit_rows)
                : static_cast<long long>(T) * a.group / unit_rows + B) * cache->Hkv;
  const long long per = (keys + piece_keys - 1) / piece_keys + (few ? kDecodeUnitCost : kChunkUnitCost);
  if (units > 0x7fffffffll / per) return FATTN_ERR_TOO_LARGE;   // the kernels number them in 32 bits
  const long long pieces = units * per;
  a.grid = pieces < max_ctas ? static_cast<int>(pieces) : max_ctas;
  CUtensorMap tk, tv;
  const long long rows = static_cast<long long>(cache->Hkv) * cache->page;
  const int box = few ? 32 : cache->page;
  if ((rc = make_rows_map_u8(&tk, cache->k, cache->d, rows, cache->pages, cache->page_stride, box)) !=
          FATTN_OK ||
      (rc = make_rows_map_u8(&tv, cache->v, cache->d, rows, cache->pages, cache->page_stride, box)) !=
          FATTN_OK)
    return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = few ? launch_cache_decode(cache->d, tk, tv, a, st)
                            : launch_cache_chunk(cache->d, tk, tv, a, st);
  return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

size_t fattn_cache_select_workspace_bytes(int T, int Hkv, int max_pages) {
  if (T <= 0 || Hkv <= 0 || Hkv > kMaxKvHeads || max_pages <= 0) return 0;
  if (cache_select_at_once(max_pages)) return 256;
  return align256(static_cast<size_t>(T) * Hkv * max_pages * sizeof(float));
}

int fattn_cache_select(const fattn_cache* cache, const void* q, long long q_row,
                       const int* page_table, const int* q_start, const int* kv_len,
                       int* selected, int n_selected, int n_first, int n_recent, void* workspace,
                       size_t workspace_bytes, int T, int B, int Hq, int max_pages,
                       fattn_stream_t stream) {
  const NvtxScope nvtx_range("fattn_cache_select");
  int rc = check_cache(cache);
  if (rc != FATTN_OK) return rc;
  if (!cache->k_bounds) return FATTN_ERR_INVALID_ARG;
  if ((rc = check_batch(cache, page_table, q_start, kv_len, T, B, max_pages)) != FATTN_OK) return rc;
  if ((rc = check_heads(cache, T, Hq)) != FATTN_OK) return rc;
  if ((rc = check_rows(q, q_row, static_cast<long long>(Hq) * cache->d)) != FATTN_OK) return rc;
  if (!selected || !aligned(selected, 4) || n_selected <= 0 || n_first < 0 || n_recent < 0 ||
      static_cast<long long>(n_first) + n_recent > n_selected)
    return FATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * cache->Hkv * n_selected > (1ll << 40)) return FATTN_ERR_INVALID_ARG;
  if (max_pages > 65535 * 128) return FATTN_ERR_INVALID_ARG;   // the grid's third extent
  const bool at_once = cache_select_at_once(max_pages);
  if (!at_once && (!workspace || !aligned(workspace, 256) ||
                   workspace_bytes < fattn_cache_select_workspace_bytes(T, cache->Hkv, max_pages)))
    return FATTN_ERR_INVALID_ARG;
  CacheSelectArgs a{};
  long long budget = 0;
  if ((rc = call_setup(&a.status, &budget)) != FATTN_OK) return rc;
  a.s = seqs_of(page_table, q_start, kv_len, T, B, max_pages);
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row;
  a.k_scale = cache->k_scale;
  a.bounds = static_cast<const int8_t*>(cache->k_bounds);
  a.pages = cache->pages;
  a.Hkv = cache->Hkv;
  a.group = Hq / cache->Hkv;
  a.page_shift = page_shift(cache->page);
  a.scores = static_cast<float*>(workspace);
  a.selected = selected;
  a.n_selected = n_selected;
  a.n_first = n_first;
  a.n_recent = n_recent;
  return launch_cache_select(cache->d, a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FATTN_OK
             : FATTN_ERR_CUDA;
}

}  // extern "C"
