// Shared by the kernels of attention over the paged latent cache: instructions,
// and how a call's tiles are dealt.
#pragma once

#include <float.h>

#include "fattn_cache.cuh"

namespace fattn {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTau = 8.f;            // a row's reference moves when a score passes it by 2^8
constexpr int kSmemMax = 232448;       // bytes a CTA may have

// P V has bf16 probabilities and the row's sum l fp32 ones, from which L comes.  O is divided by
// r, the sum of the bf16 ones, so that its weights add up to one; by l, a row that
// one key dominates would be off by that key's rounding, up to 2^-8.  A share's part of a row is
// stored as O l / r, so that parts are joined by their l alone.
// x and y plus the halves of a word.
__device__ __forceinline__ void add_bf16(float& x, float& y, uint32_t w) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(x), "+f"(y)
      : "r"(w));
}
__device__ __forceinline__ float row_factor(float l, float r, bool whole) {
  return l == 0.f ? 0.f : (whole ? 1.f : l) / r;
}

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_lead(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_lead(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// Whether a phase has completed; unlike try_wait it does not stay to see.
__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// 16 lanes x N columns: thread t gets, for each 8 columns i, r[4 i], r[4 i + 1] of
// lane t / 4, columns 8 i + 2 (t % 4) and the next, and r[4 i + 2], r[4 i + 3] of
// lane t / 4 + 8.  Valid after the wait.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// 32 lanes x 16 columns, a lane's in its thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's loads; the registers pass through, so that no use of
// them is scheduled before.
template <int K>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[K]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < K; ++i) asm volatile("" : "+r"(r[i])::"memory");
}
// Four 8 x 8 matrices of 16-bit elements, each transposed on its way.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
// A wait by a whole warp.  What comes after a first look stands once in a kernel, not at each of
// 20 to 30 places: its roles share the instruction caches, and the pieces of 1024 tokens
// take 414 us on pairs with it and 453 with the loop at each place.
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, long long budget, volatile uint32_t* abort,
                                     unsigned int site) {
  bool ok = true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) ok = false;
    else if (clock64() - t0 > budget) {
      *abort = site;
      ok = false;
    }
    if (!ok) break;
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Waits& w, unsigned int site) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_on(bar, parity, w.budget, w.abort, site);
}
__device__ __forceinline__ void prefetch_l2(const void* from, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}
// Entry `first` + lane of a sequence's row of the page table; -1 past its end.
__device__ __forceinline__ int page_of_lane(const LatentAttnArgs& a, int b, int len, int first) {
  const int p = first + static_cast<int>(threadIdx.x & 31);
  if ((static_cast<long long>(p) << a.page_shift) >= len) return -1;
  return __ldg(a.s.table + static_cast<long long>(b) * a.s.max_pages + p);
}
// ------------------------------------------------------------------ schedule

// First tile of share c of W < 2^31 dealt to G <= 152 shares: floor(W c / G).
__device__ __forceinline__ int share_first(int W, int G, int c) {
  const int q = W / G;
  return q * c + (W - q * G) * c / G;
}

// A sequence's groups of `rows` rows in order, with the key tiles that each sees.
// The tokens before the group's end, end = tok * Hq + rem, are carried along, so that
// long prompts cost no division a group.
template <int KEYS>
struct Groups {
  int rows, all;             // rows of a group and of the sequence (T * Hq < 2^31 - 1024)
  int end, tok, rem;
  int dtok, drem;
  int len, n, Hq, causal;
  __device__ __forceinline__ Groups(const LatentAttnArgs& a, const SeqInfo& q, int group_rows, int first = 0)
      : rows(group_rows), all(q.n * a.Hq), end(group_rows), len(q.len), n(q.n), Hq(a.Hq), causal(a.causal) {
    dtok = group_rows / Hq;
    drem = group_rows - dtok * Hq;
    tok = dtok;
    rem = drem;
    if (first > 0) {
      end = static_cast<int>(min(static_cast<long long>(first + 1) * group_rows, 0x7fffffffll));
      tok = end / Hq;
      rem = end - tok * Hq;
    }
  }
  __device__ __forceinline__ bool live() const { return end - rows < all; }
  __device__ __forceinline__ void next() {
    end = static_cast<int>(min(static_cast<long long>(end) + rows, 0x7fffffffll));
    tok += dtok;
    rem += drem;
    if (rem >= Hq) {
      rem -= Hq;
      ++tok;
    }
  }
  // At least one, so that rows that see nothing are written, too.
  __device__ __forceinline__ int tiles() const {
    int keys = len;
    if (causal) keys = len - n + min(n, tok + (rem > 0 ? 1 : 0));
    return max(1, (keys + KEYS - 1) / KEYS);
  }
};

// One share's part of a unit: key tiles [a, e) for row group rg of a sequence.
struct __align__(16) Seg {
  int b, rg, r0, n;
  int len, flags, a, e;
  static constexpr int kStarts = 1, kEnds = 2, kLast = 8;
  __device__ __forceinline__ bool whole() const { return (flags & 3) == 3; }
};
static_assert(sizeof(Seg) == 32, "ring slot");

// Walks a share.
template <int KEYS, int COST>
struct Walker {
  const LatentAttnArgs& a;
  int group_rows;
  int left;                 // tiles (and what units count beyond) still to walk
  int b, rg, at, nt;
  SeqInfo q;
  __device__ __forceinline__ long long all_rows() const { return static_cast<long long>(q.n) * a.Hq; }
  __device__ __forceinline__ Walker(const LatentAttnArgs& args, int rows, int first_b, int rem, int todo)
      : a(args), group_rows(rows), left(todo), b(first_b), rg(0), at(0), nt(0) {
    if (left <= 0) return;
    q = seq_info(a.s, b, a.page_shift);
    Groups<KEYS> g(a, q, group_rows);
    nt = g.tiles();
    while (rem >= nt + COST && g.live()) {
      rem -= nt + COST;
      ++rg;
      g.next();
      nt = g.tiles();
    }
    at = rem;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (left <= 0) return false;
    if (at >= nt) {                     // tiles that stand for the unit itself
      left -= nt + COST - at;
      at = 0;
      if (left <= 0) return false;
      if (static_cast<long long>(++rg) * group_rows >= all_rows()) {
        rg = 0;
        // work is left, so a sequence with rows follows
        do {
          if (++b >= a.s.B) return false;
          q = seq_info(a.s, b, a.page_shift);
        } while (q.n == 0);
      }
      nt = Groups<KEYS>(a, q, group_rows, rg).tiles();
    }
    s.b = b;
    s.rg = rg;
    s.r0 = q.r0;
    s.n = q.n;
    s.len = q.len;
    s.a = at;
    s.e = min(nt, at + left);
    s.flags = (at == 0 ? Seg::kStarts : 0) | (s.e == nt ? Seg::kEnds : 0);
    left -= s.e - s.a;
    at = s.e;
    return true;
  }
};

// A share of the call's tiles, [j0, j1) of W; `busy` shares have some.
struct Share {
  int W, busy, j0, j1;
};

// Finds share `share` of G, by all threads of a block (`side`: one number a warp in
// shared memory): place[0] is the sequence of its first tile, place[1] the tiles of
// that sequence before it, to be read behind a barrier.  `mine` has thread t's numbers
// of sequence t.
template <int KEYS, int COST, int THREADS>
__device__ __forceinline__ Share locate_share(const LatentAttnArgs& args, const SeqCheck& mine, int group_rows, int G,
                                              int share, long long* side, uint32_t* place) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (args.s.B + THREADS - 1) / THREADS;
  const int b0 = min(args.s.B, tid * per), b1 = min(args.s.B, b0 + per);
  auto info = [&](int b) {
    return b == mine.b ? seq_info(args.s, mine.r0, mine.r1, mine.len, args.page_shift)
                       : seq_info(args.s, b, args.page_shift);
  };
  auto weight = [&](const SeqInfo& q) {
    long long w = 0;
    for (Groups<KEYS> g(args, q, group_rows); g.live(); g.next()) w += g.tiles() + COST;
    return w;
  };
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqInfo q = info(b);
    if (!q.ok && blockIdx.x == 0) record_bad_index(args.status, kSiteSeqStart);
    sum += weight(q);
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  if (lane == 31) side[warp] = incl;
  __syncthreads();
  long long at = incl - sum, all = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) at += side[w];
    all += side[w];
  }
  Share s;
  s.W = total_of(all, args.status);
  s.busy = min(G, s.W);                  // no share is empty between others
  s.j0 = share < s.busy ? share_first(s.W, s.busy, share) : 0;
  s.j1 = share < s.busy ? share_first(s.W, s.busy, share + 1) : 0;
  if (s.j0 < s.j1 && at <= s.j0 && s.j0 < at + sum) {
    int b = b0;
    for (long long w; b + 1 < b1 && at + (w = weight(info(b))) <= s.j0; ++b) at += w;
    place[0] = static_cast<uint32_t>(b);
    place[1] = static_cast<uint32_t>(s.j0 - at);
    // The loader asks for the table's entries next (of a sequence's first group, here).
    const long long page = (s.j0 - at) * KEYS >> args.page_shift;
    if (page < args.s.max_pages)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(args.s.table + static_cast<long long>(b) * args.s.max_pages + page));
  }
  return s;
}

}  // namespace fattn
