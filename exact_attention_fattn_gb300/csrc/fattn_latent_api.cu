// C-ABI boundary of the paged latent cache: argument checks, tensor maps, workspace
// layout and how a call is laid out.  See include/fattn.h.
#include <math.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/fattn.h"
#include "fattn_internal.h"

namespace fattn {
namespace {

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int kMaxSeqs = 4096;
constexpr int kMaxHeads = 1024;
constexpr int kMaxSpan = 8;

int check_cache(const fattn_latent_cache* c) {
  if (!c) return FATTN_ERR_INVALID_ARG;
  if (c->rank != 256 && c->rank != 512) return FATTN_ERR_UNSUPPORTED;
  if (c->page != 32 && c->page != 64 && c->page != 128) return FATTN_ERR_UNSUPPORTED;
  if (c->pages <= 0 || !c->data || !aligned(c->data, 16)) return FATTN_ERR_INVALID_ARG;
  if (c->page_stride < static_cast<long long>(c->page) * (c->rank + kLatentRope) || c->page_stride % 8 != 0 ||
      c->page_stride >= (1ll << 38))
    return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int check_batch(const fattn_latent_cache* c, const int* page_table, const int* q_start, const int* kv_len, int T,
                int B, int max_pages) {
  if (!page_table || !q_start || !kv_len) return FATTN_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4)) return FATTN_ERR_INVALID_ARG;
  if (T <= 0 || B <= 0 || B > kMaxSeqs || max_pages <= 0) return FATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * c->page > 0x7fff0000ll) return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

// The blocks' padding rows are numbered in 32 bits, too.
int check_heads(int T, int Hq) {
  if (Hq <= 0 || Hq > kMaxHeads || static_cast<long long>(T) * Hq > 0x7fffffffll - 1024) return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int check_rows(const void* p, long long row, long long least) {
  if (!p || !aligned(p, 16) || row < least || row % 8 != 0 || row >= (1ll << 32)) return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int page_shift(int page) { return page == 32 ? 5 : (page == 64 ? 6 : 7); }

CacheSeqs seqs_of(const int* page_table, const int* q_start, const int* kv_len, int T, int B, int max_pages) {
  CacheSeqs s;
  s.q_start = q_start;
  s.kv_len = kv_len;
  s.table = page_table;
  s.T = T;
  s.B = B;
  s.max_pages = max_pages;
  return s;
}

// Rows of a block, by the rows of an average sequence (each width's products take as
// long as their 64 keys or 128 columns do, so a block has no more rows than it
// needs), and the blocks that work side by side: as few groups as blocks of kMaxSpan
// allow, and no idle block in the average sequence.
//
// Blocks of 128 rows on pairs of CTAs are for large calls of rank 512 (`reach`: keys
// that a sequence's table has room for; what they really are is on the device), a call
// in us on pairs and on single CTAs, 128 heads, one token a sequence:
//   64 of 2000 keys: 64 / 76    48 of 4000: 78 / 93    16 of 8000: 53 / 64
//   128 tokens of 64 heads on 4000: 82 / 103    8 tokens of 16 heads, 16 of 4000: 40 / 42
//   below 800 keys a pair:   16 of 1000: 27 / 24   48 of 300: 28 / 28   4 of 2000: 23 / 20
//   rows not a multiple of 128 (32 sequences of 4000 keys, 64 heads, so many tokens):
//     3: 92 / 92   5: 126 / 137   7: 157 / 184   9: 189 / 246
// For rank 256, half the products a tile, they were built and gain little, and only in the
// largest calls (32 of 8000: 61 / 63   64 of 2000: 47 / 45   16 of 1000: 22 / 17).
// Both need the same workspace, so that its size does not depend on the reach.
struct Layout {
  int rows, span;
};
Layout layout_of(int T, int B, int Hq, int rank, long long reach) {
  const long long all = (static_cast<long long>(T) * Hq + B - 1) / B, halves = (all + 63) / 64;
  const long long pairs = (halves + 1) / 2;                       // blocks of 128 rows
  Layout l;
  l.rows = all <= 16 ? 16 : (all <= 32 ? 32 : 64);
  if (rank == kLatentPairRank && (halves % 2 == 0 || halves >= 5) &&
      static_cast<double>(B) * static_cast<double>(pairs) * static_cast<double>(reach) >= 800. * (kSms / 2))
    l.rows = kLatentPairRows;
  const long long blocks = (all + l.rows - 1) / l.rows, groups = (blocks + kMaxSpan - 1) / kMaxSpan;
  l.span = static_cast<int>((blocks + groups - 1) / groups);
  return l;
}

struct Workspace {
  size_t ml_off, rec_off, total;
};
Workspace workspace_of(int rows_a_block, int rank) {
  static_assert(kSms % 2 == 0 && kLatentPairRows == 128, "pairs have the room of two blocks of 64 rows");
  Workspace w;
  const size_t rows = 2ull * kSms * (rows_a_block == kLatentPairRows ? 64 : rows_a_block);
  w.ml_off = align256(rows * rank * sizeof(float));
  w.rec_off = w.ml_off + align256(rows * sizeof(float2));
  w.total = w.rec_off + align256(kSms * sizeof(int4));
  return w;
}

}  // namespace
}  // namespace fattn

using namespace fattn;

extern "C" {

int fattn_latent_append(const fattn_latent_cache* cache, const void* latent, long long latent_row,
                        const void* k_rope, long long k_row, const void* q_rope, long long q_row,
                        long long q_head, void* q, int Hq, const float* rope, int rope_len,
                        int interleaved, const int* page_table, const int* q_start,
                        const int* kv_len, int T, int B, int max_pages, fattn_stream_t stream) {
  const Range nvtx_range("fattn_latent_append");
  int rc = check_cache(cache);
  if (rc != FATTN_OK) return rc;
  if ((rc = check_batch(cache, page_table, q_start, kv_len, T, B, max_pages)) != FATTN_OK) return rc;
  if ((rc = check_rows(latent, latent_row, cache->rank)) != FATTN_OK) return rc;
  if ((rc = check_rows(k_rope, k_row, kLatentRope)) != FATTN_OK) return rc;
  if ((q_rope == nullptr) != (q == nullptr)) return FATTN_ERR_INVALID_ARG;
  if (q_rope) {
    if ((rc = check_heads(T, Hq)) != FATTN_OK) return rc;
    if ((rc = check_rows(q_rope, q_head, kLatentRope)) != FATTN_OK) return rc;
    if ((rc = check_rows(q_rope, q_row, kLatentRope)) != FATTN_OK) return rc;
    if (!aligned(q, 16)) return FATTN_ERR_INVALID_ARG;
  }
  if (rope && (!aligned(rope, 16) || rope_len <= 0)) return FATTN_ERR_INVALID_ARG;
  LatentAppendArgs a{};
  long long budget = 0;
  if ((rc = call_setup(&a.status, &budget)) != FATTN_OK) return rc;
  a.s = seqs_of(page_table, q_start, kv_len, T, B, max_pages);
  a.data = static_cast<uint16_t*>(cache->data);
  a.page_stride = cache->page_stride;
  a.pages = cache->pages;
  a.page_shift = page_shift(cache->page);
  a.rank = cache->rank;
  a.latent = static_cast<const uint16_t*>(latent);
  a.k_rope = static_cast<const uint16_t*>(k_rope);
  a.latent_row = latent_row;
  a.k_row = k_row;
  a.q_rope = static_cast<const uint16_t*>(q_rope);
  a.qr_row = q_row;
  a.qr_head = q_head;
  a.q = static_cast<uint16_t*>(q);
  a.Hq = q_rope ? Hq : 0;
  a.rope = rope;
  a.rope_len = rope_len;
  a.interleaved = interleaved != 0;
  return launch_latent_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

size_t fattn_latent_fwd_workspace_bytes(int T, int B, int Hq, int rank) {
  if (T <= 0 || B <= 0 || B > kMaxSeqs || (rank != 256 && rank != 512) || check_heads(T, Hq) != FATTN_OK) return 0;
  return workspace_of(layout_of(T, B, Hq, rank, 0).rows, rank).total;
}

int fattn_latent_fwd(const fattn_latent_cache* cache, const void* q, void* o, float* lse,
                     const int* page_table, const int* q_start, const int* kv_len, void* workspace,
                     size_t workspace_bytes, int T, int B, int Hq, int max_pages, int causal,
                     float scale, fattn_stream_t stream) {
  const Range nvtx_range("fattn_latent_fwd");
  int rc = check_cache(cache);
  if (rc != FATTN_OK) return rc;
  if ((rc = check_batch(cache, page_table, q_start, kv_len, T, B, max_pages)) != FATTN_OK) return rc;
  if ((rc = check_heads(T, Hq)) != FATTN_OK) return rc;
  if (!q || !aligned(q, 16) || !o || !aligned(o, 16) || !lse || !aligned(lse, 4)) return FATTN_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!isfinite(scale_log2) || !(scale > 0.f)) return FATTN_ERR_INVALID_ARG;
  const Layout l = layout_of(T, B, Hq, cache->rank, static_cast<long long>(max_pages) * cache->page);
  const Workspace w = workspace_of(l.rows, cache->rank);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < w.total) return FATTN_ERR_INVALID_ARG;
  LatentAttnArgs a{};
  if ((rc = call_setup(&a.status, &a.wait_budget)) != FATTN_OK) return rc;
  a.s = seqs_of(page_table, q_start, kv_len, T, B, max_pages);
  a.data = static_cast<const uint16_t*>(cache->data);
  a.page_stride = cache->page_stride;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.pages = cache->pages;
  a.page_shift = page_shift(cache->page);
  a.Hq = Hq;
  a.causal = causal != 0;
  a.scale_log2 = scale_log2;
  char* base = static_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(base);
  a.part_ml = reinterpret_cast<float2*>(base + w.ml_off);
  a.rec = reinterpret_cast<int4*>(base + w.rec_off);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return FATTN_ERR_CUDA;
  if (sms > kSms) sms = kSms;
  // Tiles of all units, at most (the lengths are on the device).
  const long long units = static_cast<long long>(T) * Hq / (l.span * l.rows) + B;
  const bool on_pairs = l.rows == kLatentPairRows;
  const int tile = on_pairs ? kLatentPairKeys : kLatentKeys;
  const long long per = (static_cast<long long>(max_pages) * cache->page + tile - 1) / tile + latent_unit_cost(l.rows);
  if (units > 0x7fffffffll / per) return FATTN_ERR_TOO_LARGE;   // the kernels number them in 32 bits
  const long long shares = (on_pairs ? sms / 2 : sms) / l.span;
  a.span = l.span;
  a.shares = static_cast<int>(units * per < shares ? units * per : shares);
  CUtensorMap tk, tq;
  const long long width = cache->rank + kLatentRope;
  const int chunks = static_cast<int>(width / 64), box_rows = cache->page < kLatentKeys ? cache->page : kLatentKeys;
  const long long k_extents[3] = {width, cache->page, cache->pages}, k_strides[2] = {width, cache->page_stride};
  const long long q_extents[3] = {64, static_cast<long long>(T) * Hq, chunks}, q_strides[2] = {width, 64};
  const int k_box[3] = {64, box_rows, 1}, q_box[3] = {64, on_pairs ? 64 : l.rows, chunks};
  if ((rc = make_map_bf16(&tk, cache->data, 3, k_extents, k_strides, k_box)) != FATTN_OK ||
      (rc = make_map_bf16(&tq, q, 3, q_extents, q_strides, q_box)) != FATTN_OK)
    return rc;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = on_pairs ? launch_latent_pair(tk, tq, a, st)
                                 : launch_latent_attn(l.rows, cache->rank, tk, tq, a, st);
  return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}

}  // extern "C"
