// Shared by the kernels of the paged 8-bit cache: the cache's layout, the
// ragged batch that a call works on, and the checks of what the host cannot
// see (sequence starts, lengths and page numbers live on the device).
#pragma once

#include "fattn_internal.h"
#include "fattn_ptx.cuh"

namespace fattn {

constexpr unsigned int kStatusBadIndex = 7;  // == FATTN_ERR_BAD_INDEX

// What a kernel found out of range (DeviceStatus::where).
enum CacheSite : unsigned int {
  kSiteSeqStart = 401,   // q_start not ascending inside [0, T], or kv_len outside its page table
  kSitePage = 402,       // a page number outside the cache
  kSitePosition = 403,   // a new token before position 0 or past the rotation table
  kSiteSelected = 404,   // a selected page outside the page table
  kSiteRows = 405,       // a sequence that cannot be forked or freed
  kSiteRefs = 406,       // a page freed more often than it was taken, or no free page left
};

__device__ __forceinline__ void record_bad_index(DeviceStatus* st, unsigned int site) {
  if (atomicCAS(&st->code, 0u, kStatusBadIndex) == 0u) {
    st->where = site;
    st->block = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
  }
}

// Debug builds' checks of what these kernels compute (dcheck; sites 601 on).
// Every shared-memory offset lies in the launch's dynamic share, and `n` entries
// from `at` on in an array of `size`.
__device__ __forceinline__ uint32_t dynamic_smem_bytes() {
  uint32_t r;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(r));
  return r;
}
__device__ __forceinline__ bool inside(long long at, long long n, long long size) {
  return at >= 0 && at + n <= size;
}

// Waits of these kernels, as compact as they can be: the code of all of a
// CTA's roles shares the instruction caches, and a role that waits for its
// instructions holds the others up.  A wait that runs out leaves its site in
// the CTA's abort word, on which every other wait gives up; the kernel reports
// it once, at its end (report_abort).
struct Waits {
  long long budget;            // cycles
  volatile uint32_t* abort;    // shared memory
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Waits& w, unsigned int site) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*w.abort) return false;
    if (clock64() - t0 > w.budget) {
      *w.abort = site;
      return false;
    }
  }
  return true;
}

// All lanes wait; the warp goes on only if every lane saw the phase.
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, const Waits& w,
                                              unsigned int site) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, w, site));
}

__device__ __forceinline__ void report_abort(uint32_t site, DeviceStatus* st) {
  if (site != 0u && atomicCAS(&st->code, 0u, kStatusTimeout) == 0u) {
    st->where = site;
    st->block = blockIdx.x;
  }
}

// A call's kernels depend on the one before: the next is launched while that one
// runs (allow_child, on every CTA's way) and waits, in every CTA, for its end and
// for what it wrote (wait_for_parent; read with plain loads, whose order behind it
// the compiler keeps).  A call's first kernel is launched in plain stream order,
// so whatever was there before the call is complete for all of them.
__device__ __forceinline__ void allow_child() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_parent() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_child(void (*kernel)(P...), dim3 grid, dim3 block, int smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// One thread's copies (it has the barrier to itself, or its warp waits for it).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_load_1d(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// One sequence of a call: its rows [r0, r0 + n) and its cached tokens.  A
// sequence whose numbers make no sense is empty (n = len = 0), !ok.
struct SeqInfo {
  int r0, n, len;
  bool ok;
};

__device__ __forceinline__ SeqInfo seq_info(const CacheSeqs& s, int r0, int r1, int len, int page_shift) {
  SeqInfo q;
  q.r0 = r0;
  q.len = len;
  q.ok = q.r0 >= 0 && r1 >= q.r0 && r1 <= s.T && q.len >= 0 &&
         q.len <= (static_cast<long long>(s.max_pages) << page_shift);
  q.n = q.ok ? r1 - q.r0 : 0;
  if (!q.ok) q.len = 0;
  return q;
}

__device__ __forceinline__ SeqInfo seq_info(const CacheSeqs& s, int b, int page_shift) {
  return seq_info(s, __ldg(s.q_start + b), __ldg(s.q_start + b + 1), __ldg(s.kv_len + b), page_shift);
}

// Reports the sequences first, first + step, .. that make no sense.  A kernel that
// searches for its rows' or pages' sequences would otherwise miss some: where
// q_start goes back, a search passes over the sequence, and rows may seem to
// belong to none.
__device__ __forceinline__ void check_seqs(const CacheSeqs& s, int first, int step, int page_shift,
                                           DeviceStatus* st) {
  for (int b = first; b < s.B; b += step)
    if (!seq_info(s, b, page_shift).ok) record_bad_index(st, kSiteSeqStart);
}

// The same where a thread cannot wait for its first sequence's numbers: it asks
// for them at once and reports later (loads that the compiler leaves in place).
struct SeqCheck {
  int b, r0, r1, len;
  __device__ __forceinline__ SeqCheck(const CacheSeqs& s, int first) : b(first), r0(0), r1(0), len(0) {
    if (b >= s.B) return;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(r0) : "l"(s.q_start + b));
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(r1) : "l"(s.q_start + b + 1));
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(len) : "l"(s.kv_len + b));
  }
  __device__ __forceinline__ void report(const CacheSeqs& s, int step, int page_shift, DeviceStatus* st) const {
    if (b < s.B && !seq_info(s, r0, r1, len, page_shift).ok) record_bad_index(st, kSiteSeqStart);
    check_seqs(s, b + step, step, page_shift, st);
  }
};

// Pieces of work of a whole call.  The host has bounded them to 32 bits for
// sequences one behind the other; with overlapping ones the call does nothing.
__device__ __forceinline__ int total_of(long long pieces, DeviceStatus* st) {
  if (pieces <= 0x7fffffffll) return static_cast<int>(pieces);
  if (blockIdx.x == 0) record_bad_index(st, kSiteSeqStart);
  return 0;
}

// The largest b in [0, B) with f(b) <= x, f ascending, found by a whole warp
// 32 values at a time (one round of loads up to 32 sequences, two up to 1024).
// Any b in [0, B) when f is not ascending or f(0) > x.
template <class F>
__device__ __forceinline__ int find_last_warp(int B, int x, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int off = lane * step;
    const bool le = off < n && f(lo + off) <= x;
    const unsigned int m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// Work of W pieces in order, dealt to G CTAs in equal contiguous shares: the first
// piece of CTA c, and the CTA of piece j.
__device__ __forceinline__ long long cta_first(long long W, int G, int c) { return W * c / G; }
__device__ __forceinline__ int cta_of(long long W, int G, long long j) {
  return static_cast<int>(((j + 1) * G - 1) / W);
}

// 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// Exponents of the cache's scales: a scale is 2^e, kScaleExpMin <= e <= kScaleExpMax.
constexpr int kScaleExpMin = -48;
constexpr int kScaleExpMax = 48;

// log2 of a scale, whatever the memory holds: the exponent field, clamped.
__device__ __forceinline__ int scale_exp(float s) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 0xffu) - 127;
  return max(kScaleExpMin, min(kScaleExpMax, e));
}

// Four e4m3 codes -> two pairs of halves, exactly.  The 16-bit halves are
// named inside the asm: through the header's conversion, which returns a
// struct, the same two conversions ran at 8.7 instead of 21 quads a clock and SM
// (with one more operation each).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ float4 e4m3x4_to_f32x4(uint32_t codes) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(codes, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// A query row as the sum of two e4m3 rows.  `mx`: the bf16 bits of its
// largest magnitude.  The row is scaled by query_factor, a power of two, so
// that its largest entry lies in [224, 448] (448 = 1.75 * 2^8: up to 448 where the
// mantissa is at most 1.75, one power less above); query_scale undoes it.  A
// row with an infinity or a NaN becomes NaN.
__device__ __forceinline__ int query_exp(uint32_t mx) {
  const int e = static_cast<int>(mx >> 7) - 127 - 8 + ((mx & 0x7fu) > 0x60u ? 1 : 0);
  return max(-126, min(126, e));
}
__device__ __forceinline__ float query_scale(uint32_t mx) { return exp2i(query_exp(mx)); }
__device__ __forceinline__ float query_factor(uint32_t mx) {
  return mx >= 0x7f80u ? __int_as_float(0x7fffffff) : exp2i(-query_exp(mx));
}

// Four columns (two words of bf16 pairs) -> hi = e4m3(x), lo = e4m3(x - hi).  x has 8
// significant bits and hi the first 4 (rounded), so lo is exact while it is
// not subnormal and off by at most 2^-10 then.
__device__ __forceinline__ void split_query4(uint32_t p, uint32_t q, float factor, uint32_t& hi,
                                             uint32_t& lo) {
  const float x0 = __uint_as_float(p << 16) * factor, x1 = __uint_as_float(p & 0xffff0000u) * factor;
  const float x2 = __uint_as_float(q << 16) * factor, x3 = __uint_as_float(q & 0xffff0000u) * factor;
  hi = pack_e4m3x4(x0, x1, x2, x3);
  const float4 h = e4m3x4_to_f32x4(hi);
  lo = pack_e4m3x4(x0 - h.x, x1 - h.y, x2 - h.z, x3 - h.w);
}

}  // namespace fattn
