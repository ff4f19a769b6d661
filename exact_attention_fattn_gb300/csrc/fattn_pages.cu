// Pages of a cache: how often the tables name each page is counted on the
// device, and forking, growing (with a copy of a shared last page), freeing and
// compacting are kernels, so that they can be captured between the steps that
// use the pages.  A page is free while its count is zero; the lowest free pages
// are taken first, so results do not depend on timing.
//
// Bound: latency for the counts (a few integers a page; one CTA, so that the
// order needs no second launch), bytes for the copies.  A piece of a page goes through
// shared memory by two bulk copies, which one thread of a CTA issues; two CTAs an SM, six
// pieces of 16 KB each.  The list's length only the device knows.
//
// Measured: 18 of 24 sequences forked from 6 (latent cache, 300 to 4000 tokens) and
// room for one token each, both calls 14.1 us; 576 of 768 from 192 (8-bit cache, 8 heads of
// 128, 500 to 2000 tokens) and room for 100 more, 38 us; 291 MB of a pool moved together
// 58 us, 49 of them the copies, 0.87 of the measured copy rate (loads and stores of 16
// bytes a thread, 2048 threads an SM: 39 and 63.4; pieces of 24 KB 36.5 and 57.9, of
// 8 KB, with a division a piece, 58 and 75); 576 of 768 sequences of 1250 tokens freed 3.2 us.
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/fattn.h"
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kPlanes = 5;
constexpr int kMaxSeqs = 4096;
constexpr int kScanThreads = 1024;
constexpr int kScanPages = 16;          // counts a thread looks at in one turn
constexpr int kPlainThreads = 128;
constexpr int kCopyThreads = 32 + kPlainThreads;
constexpr int kStages = 6;              // pieces in shared memory, of each of two CTAs an SM
constexpr int kBehind = 2;              // of them on their way out
constexpr long long kBulkBytes = 2048;  // smaller parts of a page go by plain copies
constexpr int kPieceBytes = 16384;      // of a page's largest plane, a CTA's turn
constexpr unsigned int kStatusNoPages = FATTN_ERR_NO_PAGES;

struct Tables {
  int* table;                 // [B, max_pages]
  int B, max_pages, page_shift, pages;
  int* refs;                  // [pages]
  DeviceStatus* status;
  __device__ __forceinline__ long long cap() const { return static_cast<long long>(max_pages) << page_shift; }
  __device__ __forceinline__ int held(int len) const {
    return static_cast<int>((static_cast<long long>(len) + (1 << page_shift) - 1) >> page_shift);
  }
  __device__ __forceinline__ bool is_page(int p) const { return p >= 0 && p < pages; }
};

// What a call's second kernel copies: pages src[i] -> dst[i], i < *count.
struct CopyList {
  int* count;
  int* src;
  int* dst;
};

struct Planes {
  uint8_t* base[kPlanes];
  long long stride[kPlanes];
  long long bytes[kPlanes];
  int wide[kPlanes];          // 16-byte copies
  int bulk[kPlanes];
  int per[kPlanes];           // bytes of a piece
  int n, pieces;
};

// Exclusive prefix sum over the block of one number a thread; `total` to all.
__device__ __forceinline__ long long block_scan(long long x, long long* side, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  __syncthreads();            // side may still be read
  if (lane == 31) side[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    long long w = side[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += t;
    }
    side[lane] = w;
  }
  __syncthreads();
  total = side[31];
  return incl - x + (warp > 0 ? side[warp - 1] : 0);
}

// The counts of kScanPages pages from `first` on; pages behind the last count as
// `fill`.
__device__ __forceinline__ void load_refs(const int* refs, int pages, int first, int fill, int (&r)[kScanPages]) {
  if (first + kScanPages <= pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < kScanPages; i += 4) {
      const int4 x = *reinterpret_cast<const int4*>(refs + first + i);
      r[i] = x.x;
      r[i + 1] = x.y;
      r[i + 2] = x.z;
      r[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScanPages; ++i) r[i] = first + i < pages ? refs[first + i] : fill;
  }
}

// ------------------------------------------------------------------ fork, free

// Block i: sequence child[i] becomes a copy of parent[i], pages shared.
__global__ void __launch_bounds__(128) fork_kernel(const Tables t, int* kv_len, const int* parent, const int* child,
                                                   int n) {
  const int i = blockIdx.x;
  const int p = parent[i], c = child[i];
  bool bad = p < 0 || p >= t.B || c < 0 || c >= t.B;
  // A child is named once and is nobody's parent, so that the blocks' order does not matter.
  for (int j = threadIdx.x; j < n; j += blockDim.x) bad |= (j != i && child[j] == c) || parent[j] == c;
  bad = __syncthreads_or(bad);
  if (!bad) {
    const int len = kv_len[p];
    bad = len < 0 || len > t.cap() || kv_len[c] != 0;
    // Every thread has read kv_len[c] before one of them writes it.
    bad = __syncthreads_or(bad);
    if (!bad) {
      const int* from = t.table + static_cast<long long>(p) * t.max_pages;
      int* to = t.table + static_cast<long long>(c) * t.max_pages;
      const int held = t.held(len);
      for (int k = threadIdx.x; k < held; k += blockDim.x) {
        const int page = from[k];
        to[k] = page;
        if (t.is_page(page)) atomicAdd(t.refs + page, 1);
        else record_bad_index(t.status, kSitePage);
      }
      if (threadIdx.x == 0) kv_len[c] = len;
    }
  }
  if (bad && threadIdx.x == 0) record_bad_index(t.status, kSiteRows);
}

// Block i: sequence rows[i] gives its pages back.  Of a row named twice the first
// one counts.
__global__ void __launch_bounds__(128) free_kernel(const Tables t, int* kv_len, const int* rows, int n) {
  const int i = blockIdx.x;
  const int r = rows[i];
  if (r < 0 || r >= t.B) {
    if (threadIdx.x == 0) record_bad_index(t.status, kSiteRows);
    return;
  }
  bool twice = false;
  for (int j = threadIdx.x; j < i; j += blockDim.x) twice |= rows[j] == r;
  if (__syncthreads_or(twice)) return;
  const int len = kv_len[r];
  __syncthreads();
  if (len < 0 || len > t.cap()) {
    if (threadIdx.x == 0) record_bad_index(t.status, kSiteRows);
    return;
  }
  const int held = t.held(len);
  const int* row = t.table + static_cast<long long>(r) * t.max_pages;
  for (int k = threadIdx.x; k < held; k += blockDim.x) {
    const int page = row[k];
    if (!t.is_page(page)) {
      record_bad_index(t.status, kSitePage);
    } else if (atomicSub(t.refs + page, 1) <= 0) {
      atomicAdd(t.refs + page, 1);        // was free already
      record_bad_index(t.status, kSiteRefs);
    }
  }
  if (threadIdx.x == 0) kv_len[r] = 0;
}

// ------------------------------------------------------------------ extend

// Sequences from old_len to new_len tokens, in order: one whose next token falls
// into a page that others name too gets a copy of it, but the last of those that
// name it, if all of them write to it, keeps it; and all get the pages they lack.  Where
// the pool has too few, a sequence that needs one, or would write to a page that it
// shares, has length -1 from then on in new_len: an append that follows in the same graph,
// where no host can look in between, passes over it.
// A thread has up to kPerThread neighbouring sequences.  Whether a page's writers
// are all that name it, and which is the last, two counters a page tell (`writers`,
// `last`; sums and maxima, so their order does not matter).
constexpr int kPerThread = kMaxSeqs / kScanThreads;
constexpr int kOwnPages = 8;             // new pages that a sequence's own thread enters; more go to its warp

__global__ void __launch_bounds__(kScanThreads) extend_kernel(const Tables t, const int* old_len, int* new_len,
                                                              int* free_list, int* writers, int* last, CopyList list) {
  __shared__ long long side[32];
  __shared__ int found_all;
  const int tid = threadIdx.x, lane = tid & 31;
  allow_child();
  const int per = (t.B + kScanThreads - 1) / kScanThreads, b0 = tid * per;
  int tail[kPerThread], k0[kPerThread], k1[kPerThread], slot[kPerThread];   // shared last page, or -1; entries; the page's
  unsigned int shares = 0u;              // whether there is one
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    tail[i] = -1;
    k0[i] = k1[i] = slot[i] = 0;
    if (i >= per || b >= t.B) continue;
    const int o = old_len[b], w = new_len[b];
    if (o < 0 || w < o || w > t.cap()) {
      record_bad_index(t.status, kSiteSeqStart);
      new_len[b] = -1;
      continue;
    }
    k0[i] = t.held(o);
    k1[i] = t.held(w);
    slot[i] = o >> t.page_shift;
    if (w > o && (o & ((1 << t.page_shift) - 1)) != 0) {
      const int p = t.table[static_cast<long long>(b) * t.max_pages + slot[i]];
      if (!t.is_page(p)) record_bad_index(t.status, kSitePage);
      else if (t.refs[p] >= 2) tail[i] = p;
    }
    if (tail[i] >= 0) {
      shares |= 1u << i;
      writers[tail[i]] = 0;
      last[tail[i]] = -1;
    }
  }
  const bool shared_tails = __syncthreads_or(tail[0] >= 0 || tail[1] >= 0 || tail[2] >= 0 || tail[3] >= 0);
  static_assert(kPerThread == 4, "sequences of a thread");
  if (shared_tails) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      if (tail[i] >= 0) {
        atomicAdd(writers + tail[i], 1);
        atomicMax(last + tail[i], b0 + i);
      }
    __syncthreads();
  }
  // ---- pages that each sequence takes, copies in the upper half of the sum
  long long sum = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (tail[i] >= 0 && __ldcg(writers + tail[i]) >= t.refs[tail[i]] && __ldcg(last + tail[i]) == b0 + i) tail[i] = -1;
    sum += (tail[i] >= 0 ? (1ll << 40) + 1 : 0ll) + k1[i] - k0[i];
  }
  long long total;
  long long at = block_scan(sum, side, total);
  const long long want = total & ((1ll << 40) - 1);
  // ---- the lowest free pages
  long long seen = 0;
  if (want <= t.pages) {
    for (long long base = 0; base < t.pages && seen < want; base += kScanThreads * kScanPages) {
      int r[kScanPages], n = 0;
      const int first = static_cast<int>(min(base + tid * kScanPages, static_cast<long long>(t.pages)));
      load_refs(t.refs, t.pages, first, 1, r);
#pragma unroll
      for (int i = 0; i < kScanPages; ++i) n += r[i] == 0 ? 1 : 0;
      long long all;
      long long rank = seen + block_scan(n, side, all);
#pragma unroll
      for (int i = 0; i < kScanPages; ++i)
        if (r[i] == 0) {
          if (rank < want && dcheck(inside(rank, 1, t.pages), t.status, 671)) free_list[rank] = first + i;
          ++rank;
        }
      seen += all;
    }
  }
  if (tid == 0) found_all = seen >= want;
  __syncthreads();                       // and the list is there
  const bool granted = found_all;
  if (tid == 0) {
    *list.count = granted ? static_cast<int>(total >> 40) : 0;
    if (!granted && atomicCAS(&t.status->code, 0u, kStatusNoPages) == 0u) {
      t.status->where = kSiteRefs;
      t.status->block = 0u;
    }
  }
  // ---- copies and new entries
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    int* row = t.table + static_cast<long long>(b0 + i) * t.max_pages;
    int begin = granted ? static_cast<int>(at & ((1ll << 40) - 1)) : 0;
    const int copy = tail[i] >= 0 ? 1 : 0, fresh = k1[i] - k0[i];
    if (!granted && (fresh > 0 || (shares >> i & 1u) != 0u)) new_len[b0 + i] = -1;
    if (copy != 0 && granted) {
      const int c = static_cast<int>(at >> 40), to = free_list[begin];
      if (dcheck(inside(c, 1, t.B) && inside(begin, 1, t.pages), t.status, 672)) {
        list.src[c] = tail[i];
        list.dst[c] = to;
        row[slot[i]] = to;
        atomicSub(t.refs + tail[i], 1);
      }
      ++begin;
    }
    at += (static_cast<long long>(copy) << 40) + copy + fresh;
    if (fresh <= kOwnPages)
      for (int k = 0; k < fresh; ++k)
        if (dcheck(inside(k0[i] + k, 1, t.max_pages), t.status, 673)) row[k0[i] + k] = granted ? free_list[begin + k] : -1;
    // a warp to a sequence that takes many
    for (unsigned int many = __ballot_sync(0xffffffffu, fresh > kOwnPages); many != 0u; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const int first = __shfl_sync(0xffffffffu, k0[i], src), n = __shfl_sync(0xffffffffu, fresh, src);
      const int from = __shfl_sync(0xffffffffu, begin, src), b = __shfl_sync(0xffffffffu, b0 + i, src);
      int* to = t.table + static_cast<long long>(b) * t.max_pages + first;
      for (int k = lane; k < n; k += 32)
        if (dcheck(inside(first + k, 1, t.max_pages), t.status, 676)) to[k] = granted ? free_list[from + k] : -1;
    }
  }
  for (int i = tid; granted && i < want; i += kScanThreads) t.refs[free_list[i]] = 1;
}

// ------------------------------------------------------------------ compact

// The k-th held page from `total` on goes to the k-th free page below, total the
// number of pages held.  move_of[page]: k, for both pages of move k; other pages' entries
// hold anything, so that a reader looks whether the list has the page at that place.
// A sequence whose length makes no sense has entries that nobody could rewrite, so
// nothing moves then (limit -1).
__global__ void __launch_bounds__(kScanThreads) plan_kernel(const Tables t, const int* kv_len, int* move_of,
                                                            CopyList list, int* limit) {
  __shared__ long long side[32];
  const int tid = threadIdx.x;
  allow_child();
  bool senseless = false;
  for (int b = tid; b < t.B; b += kScanThreads) {
    const int len = kv_len[b];
    senseless |= len < 0 || len > t.cap();
  }
  // Pools of up to one turn's pages keep their counts in registers for the second look.
  const bool once = t.pages <= kScanThreads * kScanPages;
  int r[kScanPages];
  long long held = 0;
  for (long long base = 0; base < t.pages; base += kScanThreads * kScanPages) {
    load_refs(t.refs, t.pages, static_cast<int>(min(base + tid * kScanPages, static_cast<long long>(t.pages))), 0, r);
#pragma unroll
    for (int i = 0; i < kScanPages; ++i) held += r[i] > 0 ? 1 : 0;
  }
  if (__syncthreads_or(senseless)) {
    if (tid == 0) {
      record_bad_index(t.status, kSiteSeqStart);
      *list.count = 0;
      *limit = -1;
    }
    return;
  }
  long long total;
  block_scan(held, side, total);
  long long seen = 0;                    // holes, and pages to move in the upper half
  for (long long base = 0; base < t.pages; base += kScanThreads * kScanPages) {
    const int first = static_cast<int>(min(base + tid * kScanPages, static_cast<long long>(t.pages)));
    if (!once) load_refs(t.refs, t.pages, first, 0, r);
    long long n = 0;
#pragma unroll
    for (int i = 0; i < kScanPages; ++i) {
      const int p = first + i;
      if (p < total && r[i] <= 0) n += 1;
      if (p >= total && r[i] > 0) n += 1ll << 32;
    }
    long long all;
    const long long at = seen + block_scan(n, side, all);
    int hole = static_cast<int>(at & 0xffffffffll), move = static_cast<int>(at >> 32);
#pragma unroll
    for (int i = 0; i < kScanPages; ++i) {
      const int p = first + i;
      if (!dcheck(hole <= t.pages / 2 && move <= t.pages / 2, t.status, 674)) break;
      if (p < total && p < t.pages && r[i] <= 0) list.dst[hole++] = p;
      if (p >= total && r[i] > 0) list.src[move++] = p;
    }
    seen += all;
  }
  __syncthreads();
  const int moves = static_cast<int>(seen >> 32);
  for (int i = tid; i < moves; i += kScanThreads) {
    const int from = list.src[i], to = list.dst[i];
    move_of[from] = move_of[to] = i;
    t.refs[to] = t.refs[from];
    t.refs[from] = 0;
  }
  if (tid == 0) {
    *list.count = moves;
    *limit = static_cast<int>(total);
  }
}

// ------------------------------------------------------------------ copies

// A group of its own; all but the last kBehind groups have then read their source.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile(
      "cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\t"
      "cp.async.bulk.commit_group;\n\t"
      "cp.async.bulk.wait_group.read %3;" ::"l"(dst),
      "r"(src), "r"(bytes), "n"(kBehind)
      : "memory");
}
__device__ __forceinline__ void bulk_wait_group0() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <class V>
__device__ __forceinline__ void copy_span(uint8_t* to, const uint8_t* from, long long bytes, int thread) {
  const V* s = reinterpret_cast<const V*>(from);
  V* d = reinterpret_cast<V*>(to);
  const int n = static_cast<int>(bytes / sizeof(V));
  for (int i = thread; i < n; i += kPlainThreads) d[i] = s[i];
}

// Piece `piece` of plane k of a page: its first byte and its length, which may be 0.
__device__ __forceinline__ int piece_of(const Planes& p, int k, int piece, long long& lo) {
  lo = min(p.bytes[k], static_cast<long long>(piece) * p.per[k]);
  return static_cast<int>(min(p.bytes[k], lo + p.per[k]) - lo);
}

// Copies the list's pages and, where kv_len is given, rewrites the table where pages have
// moved (compact).  One thread moves a CTA's pieces through shared memory by bulk copies,
// kStages - kBehind on their way in; the others take what is small or not aligned to
// 16 bytes, and the table.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const Tables t, const __grid_constant__ Planes planes,
                                                            CopyList list, const int* kv_len, const int* move_of,
                                                            const int* limit, long long wait_budget) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ uint64_t full[kStages];
  __shared__ uint8_t* out[kStages];
  __shared__ uint32_t length[kStages];
  __shared__ uint32_t abort;
  const uint32_t sbase = smem_u32(stages);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&full[i]), 1);
    fence_barrier_init();
    abort = 0u;
  }
  wait_for_parent();
  const int n = *list.count;
  if (n == 0 && kv_len == nullptr) return;
  const long long items = static_cast<long long>(n) * planes.pieces;
  if (threadIdx.x >= 32) {
    const int me = threadIdx.x - 32;
    for (long long w = blockIdx.x; w < items; w += gridDim.x) {
      const int i = static_cast<int>(w / planes.pieces), piece = static_cast<int>(w - static_cast<long long>(i) * planes.pieces);
      for (int k = 0; k < planes.n; ++k) {
        if (planes.bulk[k]) continue;
        const long long from = list.src[i], to = list.dst[i];
        if (!dcheck(inside(from, 1, t.pages) && inside(to, 1, t.pages), t.status, 675)) continue;
        long long lo;
        const int span = piece_of(planes, k, piece, lo);
        uint8_t* d = planes.base[k] + to * planes.stride[k] + lo;
        const uint8_t* s = planes.base[k] + from * planes.stride[k] + lo;
        if (planes.wide[k]) copy_span<uint4>(d, s, span, me);
        else copy_span<uint32_t>(d, s, span, me);
      }
    }
    if (kv_len == nullptr) return;
    const int lim = *limit;
    if (lim < 0) return;
    for (int b = blockIdx.x; b < t.B; b += gridDim.x) {
      int* row = t.table + static_cast<long long>(b) * t.max_pages;
      const int held = t.held(kv_len[b]);
      for (int k = me; k < held; k += kPlainThreads) {
        const int p = row[k];
        if (!t.is_page(p)) {
          record_bad_index(t.status, kSitePage);
          continue;
        }
        // From the limit on only pages that moved were held, and below it those that were
        // moved to were not: such an entry stays, and is reported.
        const int i = move_of[p];
        const bool listed = i >= 0 && i < n && (p >= lim ? list.src : list.dst)[i] == p;
        if (listed != (p >= lim)) record_bad_index(t.status, kSiteRefs);
        else if (listed) row[k] = list.dst[i];
      }
    }
    return;
  }
  if (threadIdx.x != 0) return;
  // The next piece to load, of page i's planes from k on; the numbers of the page after
  // it are asked for a turn early.
  const int pages_on = gridDim.x / planes.pieces, pieces_on = gridDim.x - pages_on * planes.pieces;
  int i = blockIdx.x / planes.pieces, piece = blockIdx.x - i * planes.pieces, k = 0;
  int next_from = i < n ? list.src[i] : 0, next_to = i < n ? list.dst[i] : 0;
  long long from = 0, to = 0;
  bool fresh = true;
  auto next = [&](const uint8_t*& src, uint8_t*& dst) -> uint32_t {
    while (i < n) {
      if (fresh) {
        from = next_from;
        to = next_to;
        const int ahead = i + pages_on + (piece + pieces_on >= planes.pieces ? 1 : 0);
        if (ahead < n) {
          next_from = list.src[ahead];
          next_to = list.dst[ahead];
        }
        fresh = false;
        k = dcheck(inside(from, 1, t.pages) && inside(to, 1, t.pages), t.status, 677) ? 0 : planes.n;
      }
      while (k < planes.n) {
        const int p = k++;
        if (!planes.bulk[p]) continue;
        long long lo;
        const int span = piece_of(planes, p, piece, lo);
        if (span == 0 || !dcheck(span <= kPieceBytes, t.status, 678)) continue;
        src = planes.base[p] + from * planes.stride[p] + lo;
        dst = planes.base[p] + to * planes.stride[p] + lo;
        return static_cast<uint32_t>(span);
      }
      i += pages_on;
      piece += pieces_on;
      if (piece >= planes.pieces) {
        piece -= planes.pieces;
        ++i;
      }
      fresh = true;
    }
    return 0u;
  };
  const WaitCtx wc{wait_budget, &abort, t.status};
  unsigned int loads = 0, stores = 0;
  bool more = true;
  while (true) {
    // A stage is free once the store from it has read it: all but the last kBehind have.
    while (more && loads - (stores > kBehind ? stores - kBehind : 0u) < kStages) {
      const uint8_t* src = nullptr;
      const unsigned int at = loads % kStages;
      const uint32_t bytes = next(src, out[at]);
      if (!(more = bytes != 0u)) break;
      length[at] = bytes;
      mbar_arrive_expect_tx(smem_u32(&full[at]), bytes);
      bulk_load_1d(sbase + at * kPieceBytes, src, bytes, smem_u32(&full[at]));
      ++loads;
    }
    if (stores == loads) break;
    const unsigned int at = stores % kStages;
    if (!mbar_wait(smem_u32(&full[at]), (stores / kStages) & 1, wc, kWaitKvFull)) break;
    bulk_store(out[at], sbase + at * kPieceBytes, length[at]);
    ++stores;
  }
  bulk_wait_group0();
  for (; stores < loads; ++stores) mbar_wait_drain(smem_u32(&full[stores % kStages]), (stores / kStages) & 1);
}

// ------------------------------------------------------------------ host

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_pool(const fattn_page_pool* pool, const int* page_table, const int* kv_len, int B, int max_pages) {
  if (!pool || !pool->refs || !aligned(pool->refs, 4) || pool->pages <= 0) return FATTN_ERR_INVALID_ARG;
  if (pool->page != 32 && pool->page != 64 && pool->page != 128) return FATTN_ERR_UNSUPPORTED;
  if (!page_table || !kv_len || !aligned(page_table, 4) || !aligned(kv_len, 4)) return FATTN_ERR_INVALID_ARG;
  if (B <= 0 || B > kMaxSeqs || max_pages <= 0) return FATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * pool->page > 0x7fff0000ll || pool->pages >= (1 << 30))
    return FATTN_ERR_INVALID_ARG;
  return FATTN_OK;
}

int check_planes(const fattn_page_pool* pool, const fattn_plane* planes, int n, Planes& out) {
  if (!planes || n <= 0 || n > kPlanes) return FATTN_ERR_INVALID_ARG;
  long long most = 0;
  for (int i = 0; i < n; ++i) {
    const fattn_plane& p = planes[i];
    if (!p.base || !aligned(p.base, 4) || p.bytes <= 0 || p.bytes % 4 != 0 || p.stride % 4 != 0 ||
        p.stride < p.bytes || p.stride >= (1ll << 40) || p.bytes > 0x7fffffffll)
      return FATTN_ERR_INVALID_ARG;
    out.base[i] = static_cast<uint8_t*>(p.base);
    out.stride[i] = p.stride;
    out.bytes[i] = p.bytes;
    out.wide[i] = aligned(p.base, 16) && p.bytes % 16 == 0 && p.stride % 16 == 0;
    out.bulk[i] = out.wide[i] && p.bytes >= kBulkBytes;
    most = p.bytes > most ? p.bytes : most;
  }
  (void)pool;
  out.n = n;
  out.pieces = static_cast<int>((most + kPieceBytes - 1) / kPieceBytes);
  for (int i = 0; i < n; ++i) {
    const long long unit = out.wide[i] ? 16 : 4;
    out.per[i] = static_cast<int>((out.bytes[i] / unit + out.pieces - 1) / out.pieces * unit);
  }
  return FATTN_OK;
}

Tables tables_of(const fattn_page_pool* pool, int* page_table, int B, int max_pages, DeviceStatus* status) {
  Tables t;
  t.table = page_table;
  t.B = B;
  t.max_pages = max_pages;
  t.page_shift = pool->page == 32 ? 5 : (pool->page == 64 ? 6 : 7);
  t.pages = pool->pages;
  t.refs = pool->refs;
  t.status = status;
  return t;
}

// count and limit, then two lists of pages, then three numbers a page
struct PagesWorkspace {
  size_t src, dst, map, writers, last, total;
};
PagesWorkspace workspace_of(int pages, int B) {
  PagesWorkspace w;
  const size_t list = align256((static_cast<size_t>(pages / 2 > B ? pages / 2 : B) + 1) * sizeof(int));
  w.src = 256;
  w.dst = w.src + list;
  w.map = w.dst + list;
  const size_t each = align256(static_cast<size_t>(pages) * sizeof(int));
  w.writers = w.map + each;
  w.last = w.writers + each;
  w.total = w.last + each;
  return w;
}

int launch_copies(const Tables& t, const Planes& p, const CopyList& list, long long most_pages, const int* kv_len,
                  const int* move_of, const int* limit, long long budget, cudaStream_t stream) {
  static SmemLimit limit_of;
  constexpr int kBytes = kStages * kPieceBytes;
  if (limit_of.raise(reinterpret_cast<const void*>(copy_kernel), kBytes) != cudaSuccess) return FATTN_ERR_CUDA;
  const long long items = most_pages * p.pieces;
  const int grid = static_cast<int>(items < 2 * kSms ? items : 2 * kSms);
  return launch_child(copy_kernel, grid, kCopyThreads, kBytes, stream, t, p, list, kv_len, move_of, limit, budget) ==
                 cudaSuccess
             ? FATTN_OK
             : FATTN_ERR_CUDA;
}

int from_launch(cudaError_t e) { return e == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA; }

}  // namespace

}  // namespace fattn

using namespace fattn;

extern "C" {

int fattn_pages_fork(const fattn_page_pool* pool, int* page_table, int* kv_len, const int* parent, const int* child,
                     int n, int B, int max_pages, fattn_stream_t stream) {
  const Range range("fattn_pages_fork");
  int rc = check_pool(pool, page_table, kv_len, B, max_pages);
  if (rc != FATTN_OK) return rc;
  if (!parent || !child || !aligned(parent, 4) || !aligned(child, 4) || n <= 0 || n > B) return FATTN_ERR_INVALID_ARG;
  DeviceStatus* status = nullptr;
  long long budget = 0;
  if ((rc = call_setup(&status, &budget)) != FATTN_OK) return rc;
  fork_kernel<<<n, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(tables_of(pool, page_table, B, max_pages, status),
                                                                     kv_len, parent, child, n);
  return from_launch(cudaGetLastError());
}

int fattn_pages_free(const fattn_page_pool* pool, int* page_table, int* kv_len, const int* rows, int n, int B,
                     int max_pages, fattn_stream_t stream) {
  const Range range("fattn_pages_free");
  int rc = check_pool(pool, page_table, kv_len, B, max_pages);
  if (rc != FATTN_OK) return rc;
  if (!rows || !aligned(rows, 4) || n <= 0 || n > kMaxSeqs) return FATTN_ERR_INVALID_ARG;
  DeviceStatus* status = nullptr;
  long long budget = 0;
  if ((rc = call_setup(&status, &budget)) != FATTN_OK) return rc;
  free_kernel<<<n, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(tables_of(pool, page_table, B, max_pages, status),
                                                                     kv_len, rows, n);
  return from_launch(cudaGetLastError());
}

size_t fattn_pages_workspace_bytes(int pages, int B) {
  if (pages <= 0 || pages >= (1 << 30) || B <= 0 || B > kMaxSeqs) return 0;
  return workspace_of(pages, B).total;
}

int fattn_pages_extend(const fattn_page_pool* pool, const fattn_plane* planes, int n_planes, int* page_table,
                       const int* old_len, int* new_len, void* workspace, size_t workspace_bytes, int B,
                       int max_pages, fattn_stream_t stream) {
  const Range range("fattn_pages_extend");
  int rc = check_pool(pool, page_table, old_len, B, max_pages);
  if (rc != FATTN_OK) return rc;
  if (!new_len || !aligned(new_len, 4)) return FATTN_ERR_INVALID_ARG;
  Planes p{};
  if ((rc = check_planes(pool, planes, n_planes, p)) != FATTN_OK) return rc;
  const PagesWorkspace w = workspace_of(pool->pages, B);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < w.total) return FATTN_ERR_INVALID_ARG;
  DeviceStatus* status = nullptr;
  long long budget = 0;
  if ((rc = call_setup(&status, &budget)) != FATTN_OK) return rc;
  char* base = static_cast<char*>(workspace);
  const CopyList list{reinterpret_cast<int*>(base), reinterpret_cast<int*>(base + w.src),
                      reinterpret_cast<int*>(base + w.dst)};
  const Tables t = tables_of(pool, page_table, B, max_pages, status);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  extend_kernel<<<1, kScanThreads, 0, st>>>(t, old_len, new_len, reinterpret_cast<int*>(base + w.map),
                                          reinterpret_cast<int*>(base + w.writers),
                                          reinterpret_cast<int*>(base + w.last), list);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return FATTN_ERR_CUDA;
  return launch_copies(t, p, list, B, nullptr, nullptr, nullptr, budget, st);
}

int fattn_pages_compact(const fattn_page_pool* pool, const fattn_plane* planes, int n_planes, int* page_table,
                        const int* kv_len, void* workspace, size_t workspace_bytes, int B, int max_pages,
                        fattn_stream_t stream) {
  const Range range("fattn_pages_compact");
  int rc = check_pool(pool, page_table, kv_len, B, max_pages);
  if (rc != FATTN_OK) return rc;
  Planes p{};
  if ((rc = check_planes(pool, planes, n_planes, p)) != FATTN_OK) return rc;
  const PagesWorkspace w = workspace_of(pool->pages, B);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < w.total) return FATTN_ERR_INVALID_ARG;
  DeviceStatus* status = nullptr;
  long long budget = 0;
  if ((rc = call_setup(&status, &budget)) != FATTN_OK) return rc;
  char* base = static_cast<char*>(workspace);
  const CopyList list{reinterpret_cast<int*>(base), reinterpret_cast<int*>(base + w.src),
                      reinterpret_cast<int*>(base + w.dst)};
  int* limit = reinterpret_cast<int*>(base) + 1;
  int* move_of = reinterpret_cast<int*>(base + w.map);
  const Tables t = tables_of(pool, page_table, B, max_pages, status);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  plan_kernel<<<1, kScanThreads, 0, st>>>(t, kv_len, move_of, list, limit);
  if (cudaGetLastError() != cudaSuccess) return FATTN_ERR_CUDA;
  return launch_copies(t, p, list, static_cast<long long>(pool->pages) / 2 + 1, kv_len, move_of, limit, budget, st);
}

}  // extern "C"
