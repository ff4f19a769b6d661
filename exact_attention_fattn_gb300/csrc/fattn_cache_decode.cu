// Attention over the paged 8-bit cache for few query rows per sequence
// (single tokens, short drafts).
//
// The rows of a unit -- up to 16 (token, query head) pairs of one sequence
// that share a kv head -- meet every cached key of that head once, so the
// call is bound by reading the cache, 2 d bytes a token and kv head.  With
// 16 rows or fewer a 128-row tcgen05 tile would be mostly padding; the
// products go to mma.sync m16n8k16 in fp16 (measured on GB300: 8 cycles each
// per SM quarter, 512 per 128 keys and SM, where the memory needs 1400).
//
// Codes become halves in registers: an e4m3 value is exact in fp16.  Queries
// are scaled by a power of two per row into fp16's range, exactly unless an
// entry is 2^-14 below its row's largest; probabilities are rounded to fp16
// (11 bits) for P V and summed in fp32 unrounded.  (mma.sync on the codes
// themselves, with Q in two e4m3 parts, is 20 % slower: the compiler converts
// both operands in front of every such product.)
//
// Softmax with the value scales inside: with sv_p the value scale of page p
// and l_p its log2,
//   x_j = s_j + l_p(j),  m = running max of x - 14,  P'_j = 2^(x_j - m),
//   O = sum P'_j V8_j,   l = sum_p 2^(-l_p) sum_{j in p} P'_j,
// so O / l is the result and m + log2 l the log-sum-exp, with one exponential
// per score and no product by the scales left over; |l_p| <= 48 keeps the sum
// in range.  With the reference 14 below the maximum fp16 holds probabilities
// down to 2^-38 of the largest, so that many small ones are not lost.
//
// Work split: a unit's keys are cut into chunks of 128 and the chunks of all
// units, in order, are dealt to the CTAs in equal contiguous shares, so
// lengths may differ by any factor.  A unit counts two pieces more than it has
// chunks, about what beginning and ending it costs, so that CTAs with many
// short units end with the others (64 sequences of 500 to 8000 tokens, 8 kv heads
// of 128: 108 us without them, 103 with one, 101 with two and with three).  A
// CTA's 4 warps take 32 keys of each chunk, each with its own softmax state and its own ring of TMA tiles (no
// barrier inside a chunk), and are joined through shared memory when the
// CTA's part of the unit ends; the next unit's queries are on their way to
// shared memory by then, and the SM's other CTAs work meanwhile.  A unit that
// several CTAs share is joined from their partial results in a second
// kernel, in order, so results do not depend on timing.
//
// Measured on GB300, join included: that batch 99 us (5.7 TB/s, 0.84 of the
// copy rate), 2 x up to 131071 tokens 80 us (0.86), one sequence of 1000 tokens 12.3
// us (latency: two launches and five dependent loads).  What is left of the large
// calls is the first 6 us, before the copies flow, and the join.
#include <cuda_fp16.h>

#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = kDecodeRows;
constexpr int kTileKeys = 32;                       // keys a warp takes of a chunk
constexpr int kChunkKeys = kWarps * kTileKeys;
static_assert(kChunkKeys == kDecodeKeys, "pieces of work");
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLift = 14.f;                       // log2 of the largest P' (fp16 holds 65504)

template <int D>
struct DecCfg {
  static constexpr int kTileBytes = kTileKeys * D;  // K or V of a tile
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // A warp's rows of O at the end of a unit go where its last tile was.
  static_assert(kRows * D * 4 <= kStageBytes, "a stage holds a warp's O");
  static constexpr int kMlOff = kRingBytes;         // [kWarps][kRows] float2
  static constexpr int kQOff = kMlOff + kWarps * kRows * 8;           // [2][kRows][D] bf16
  static constexpr int kBarOff = kQOff + 2 * kRows * D * 2;
  static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;     // abort, then two units
  static constexpr int kPreOff = kMiscOff + 128;    // [B + 1] int
  static constexpr int kSmemFixed = kPreOff + 1024;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Chunks of a unit: at least one, so that rows that see nothing are written.
__device__ __forceinline__ int chunks_of(int len) {
  return max(1, (len + kChunkKeys - 1) / kChunkKeys);
}

// A unit: rows [16 rb, ..) of a sequence's n * group rows, one kv head.
// Sparse calls take each token as a sequence of its own (r0 = token, n = 1).
struct Unit {
  int seq;            // sequence, sparse: token
  int rb, head;
  int r0, n;          // rows of the call
  int pos0;           // position of row r0
  int len;            // keys that exist
  int table_row;      // row of the page table
  int c0, chunks;     // first piece of work, and chunks; pieces() with what the unit itself costs
  __device__ __forceinline__ int pieces(bool sparse) const {
    return chunks + (sparse ? 0 : kDecodeUnitCost);   // sparse units all have the same number
  }
};

__device__ __forceinline__ Unit shfl_unit(Unit u) {   // lane 0's, as far as queries need it
  u.rb = __shfl_sync(0xffffffffu, u.rb, 0);
  u.head = __shfl_sync(0xffffffffu, u.head, 0);
  u.r0 = __shfl_sync(0xffffffffu, u.r0, 0);
  u.n = __shfl_sync(0xffffffffu, u.n, 0);
  return u;
}

// Pieces of work of the whole call, and the unit of a piece.  pre: dense calls
// only, pieces before each sequence (shared memory, [B + 1]).
struct Schedule {
  const CacheAttnArgs* a;
  const int* pre;
  int sparse_chunks;      // chunks of every sparse unit
  int sparse_blocks;      // row blocks of a token's group

  __device__ __forceinline__ int total() const {
    return a->selected != nullptr ? a->s.T * a->Hkv * sparse_blocks * sparse_chunks : pre[a->s.B];
  }
  __device__ __forceinline__ Unit sequence(int b) const {
    const SeqInfo q = seq_info(a->s, b, a->page_shift);
    Unit u;
    u.seq = u.table_row = b;
    u.rb = u.head = 0;
    u.r0 = q.r0;
    u.n = q.n;
    u.len = q.len;
    u.pos0 = q.len - q.n;
    u.c0 = pre[b];
    u.chunks = chunks_of(q.len);
    return u;
  }
  __device__ __forceinline__ Unit unit_of(int j) const {
    if (a->selected != nullptr) {
      Unit u;
      const int id = j / sparse_chunks, hb = id / a->Hkv;
      u.c0 = id * sparse_chunks;
      u.chunks = sparse_chunks;
      u.head = id - hb * a->Hkv;
      u.rb = hb % sparse_blocks;
      u.seq = hb / sparse_blocks;
      finish(u);
      return u;
    }
    int lo = 0, hi = a->s.B;   // the last b with pre[b] <= j
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= j) lo = mid; else hi = mid;
    }
    Unit u = sequence(lo);
    const int id = (j - u.c0) / u.pieces(false);
    u.c0 += id * u.pieces(false);
    u.rb = id / a->Hkv;
    u.head = id - u.rb * a->Hkv;
    return u;
  }
  // The unit after u; there is one.
  __device__ __forceinline__ void advance(Unit& u) const {
    u.c0 += u.pieces(a->selected != nullptr);
    if (++u.head < a->Hkv) return;
    u.head = 0;
    ++u.rb;
    if (a->selected != nullptr) {
      if (u.rb < sparse_blocks) return;
      u.rb = 0;
      ++u.seq;
      finish(u);
      return;
    }
    if (u.rb * kRows < u.n * a->group) return;
    int b = u.seq;
    while (b + 1 < a->s.B && pre[b + 1] == pre[b + 2]) ++b;   // sequences without rows
    u = sequence(min(b + 1, a->s.B - 1));
  }
  // The sequence of a sparse unit's token: a guess that holds where all
  // sequences have the same number of rows, else a search.
  __device__ __forceinline__ void finish(Unit& u) const {
    u.r0 = u.seq;
    const int* qs = a->s.q_start;
    int b = static_cast<int>(static_cast<long long>(u.r0) * a->s.B / a->s.T);
    if (u.r0 < __ldg(qs + b) || u.r0 >= __ldg(qs + b + 1)) {
      b = 0;
      for (int hi = a->s.B; hi - b > 1;) {
        const int mid = (b + hi) >> 1;
        if (__ldg(qs + mid) <= u.r0) b = mid; else hi = mid;
      }
    }
    const SeqInfo q = seq_info(a->s, b, a->page_shift);
    if (!q.ok) record_bad_index(a->status, kSiteSeqStart);
    u.table_row = b;
    if (u.r0 < q.r0 || u.r0 >= q.r0 + q.n) {
      u.n = 0;     // a row behind the last sequence
      u.len = u.pos0 = 0;
      return;
    }
    u.n = 1;
    u.pos0 = q.len - q.n + (u.r0 - q.r0);
    u.len = a->causal ? max(0, min(q.len, u.pos0 + 1)) : q.len;
  }
};

// One tile of a warp, as lane i of a batch of 32 looks it up.
struct Tile {
  int pid;        // page, or -1: nothing to read
  int y;          // row of the page's [Hkv * page] rows
  int key0;       // position of its first key
  float ks;       // K scale
  float vs;       // V scale
};

__device__ __forceinline__ Tile shfl_tile(const Tile& t, int src) {
  Tile r;
  r.pid = __shfl_sync(0xffffffffu, t.pid, src);
  r.y = __shfl_sync(0xffffffffu, t.y, src);
  r.key0 = __shfl_sync(0xffffffffu, t.key0, src);
  r.ks = __shfl_sync(0xffffffffu, t.ks, src);
  r.vs = __shfl_sync(0xffffffffu, t.vs, src);
  return r;
}

template <int D, bool SPARSE>
__global__ void __launch_bounds__(kThreads, decode_ctas(D))
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CacheAttnArgs a) {
  using C = DecCfg<D>;
  constexpr int kK = D / 16;            // k steps of Q K^T
  constexpr int kVals = D / 4;          // consecutive columns of O a thread holds per row
  constexpr int kTiles8 = kVals / 2;    // n8 tiles of P V
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  float2* ml = reinterpret_cast<float2*>(smem + C::kMlOff);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  int* pre = reinterpret_cast<int*>(smem + C::kPreOff);
  Unit* units = reinterpret_cast<Unit*>(smem + C::kMiscOff + 16);   // this one and the next
  static_assert(sizeof(Unit) * 2 + 16 <= 128, "two units");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const uint32_t ring = sbase + warp * C::kStages * C::kStageBytes;
  const uint32_t bar0 = sbase + C::kBarOff + warp * C::kStages * 8;
  const int G = a.grid, cta = blockIdx.x;
  [[maybe_unused]] constexpr long long kPartRows = part_rows(D, kRows);
  if (!dcheck(smem_u32(pre + (SPARSE ? 0 : a.s.B + 1)) <= smem_u32(smem_raw) + dynamic_smem_bytes() &&
                  2ll * (cta + 1) * kRows <= kPartRows,
              a.status, 631))
    return;

  // a sparse call searches for its tokens' sequences only (in the join's
  // kernel this check cost 0.6 us of 39)
  const SeqCheck check(a.s, SPARSE ? cta * kThreads + tid : a.s.B);
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (tid == 0) misc[0] = 0u;
  fence_barrier_init();

  // ---- pieces of work before each sequence
  if constexpr (!SPARSE) {
    const int per = (a.s.B + kThreads - 1) / kThreads;
    const int b0 = min(a.s.B, tid * per), b1 = min(a.s.B, b0 + per);
    // 64 bits: sequences whose rows overlap may need more than the call can
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const SeqInfo q = seq_info(a.s, b, a.page_shift);
      if (!q.ok && cta == 0) record_bad_index(a.status, kSiteSeqStart);
      pre[b] = static_cast<int>(sum);
      sum += static_cast<long long>((q.n * a.group + kRows - 1) / kRows) * a.Hkv *
             (chunks_of(q.len) + kDecodeUnitCost);
    }
    long long incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += t;
    }
    long long* wtot = reinterpret_cast<long long*>(ml);
    if (lane == 31) wtot[warp] = incl;
    __syncthreads();
    long long at = incl - sum;
    for (int w = 0; w < warp; ++w) at += wtot[w];
    for (int b = b0; b < b1; ++b) pre[b] += static_cast<int>(at);
    if (tid == kThreads - 1) pre[a.s.B] = total_of(at + sum, a.status);
  }
  __syncthreads();

  const Schedule sched{&a, pre, SPARSE ? ((a.n_selected << a.page_shift) + kChunkKeys - 1) / kChunkKeys : 0,
                       (a.group + kRows - 1) / kRows};
  const int W = sched.total();
  const int j0 = static_cast<int>(cta_first(W, G, cta)), j1 = static_cast<int>(cta_first(W, G, cta + 1));
  const int n_tiles = j1 - j0;                      // of this warp, and of every other
  const Waits wc{a.wait_budget, reinterpret_cast<volatile uint32_t*>(&misc[0])};

  // A unit's queries into shared memory, rows past its last as zeros.
  auto fetch_q = [&](const Unit& u, int buf) {
    for (int x = tid; x < kRows * (D / 8); x += kThreads) {
      const int row = x / (D / 8), col = x % (D / 8), rr = u.rb * kRows + row;
      const bool on = rr < u.n * a.group;
      const int token = on ? rr / a.group : 0;
      const uint16_t* src = a.q + (u.r0 + token) * a.q_row +
                            (static_cast<long long>(u.head) * a.group + (on ? rr - token * a.group : 0)) * D + 8 * col;
      const uint32_t dst = sbase + C::kQOff + ((buf * kRows + row) * D + 8 * col) * 2;
      if (!dcheck(in_range(dst, 16, sbase + C::kQOff, sbase + C::kBarOff) &&
                      (!on || (inside(u.r0 + token, 1, a.s.T) && inside(u.head, 1, a.Hkv))),
                  a.status, 632))
        continue;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(on ? src : a.q),
                   "r"(on ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // The tiles of pieces j0 + 32 k .. + 31, one per lane, and their units.
  auto look_up = [&](int k, Unit& u) -> Tile {
    Tile t{-1, 0, 0, 0.f, 0.f};
    const int i = 32 * k + lane;
    if (i >= n_tiles) return t;
    u = sched.unit_of(j0 + i);
    if (u.n == 0 || j0 + i - u.c0 >= u.chunks) return t;
    const int at = (j0 + i - u.c0) * kChunkKeys + warp * kTileKeys;
    const int page = 1 << a.page_shift;
    int entry = at >> a.page_shift;
    const int off = at & (page - 1);
    if constexpr (SPARSE) {
      if (entry >= a.n_selected) return t;
      entry = __ldg(a.selected + (static_cast<long long>(u.seq) * a.Hkv + u.head) * a.n_selected + entry);
      if (entry < 0) return t;
      if (entry >= a.s.max_pages) {
        record_bad_index(a.status, kSiteSelected);
        return t;
      }
    }
    const long long key0 = (static_cast<long long>(entry) << a.page_shift) + off;
    if (key0 >= u.len) return t;
    const int pid = __ldg(a.s.table + static_cast<long long>(u.table_row) * a.s.max_pages + entry);
    if (pid < 0 || pid >= a.pages) {
      record_bad_index(a.status, kSitePage);
      return t;
    }
    t.pid = pid;
    t.y = u.head * page + off;
    t.key0 = static_cast<int>(key0);
    const long long sc = static_cast<long long>(pid) * a.Hkv + u.head;
    t.ks = __ldg(a.k_scale + sc);
    t.vs = __ldg(a.v_scale + sc);
    return t;
  };
  // Tile `src` of a batch into a stage (converged warp): whether there is one.
  auto issue = [&](const Tile& batch, int src, int stage) -> bool {
    const int pid = __shfl_sync(0xffffffffu, batch.pid, src);
    const int y = __shfl_sync(0xffffffffu, batch.y, src);
    if (pid < 0) return false;
    if (!dcheck(stage >= 0 && in_range(ring + stage * C::kStageBytes, C::kStageBytes, sbase, sbase + C::kRingBytes) &&
                    pid < a.pages && inside(y, kTileKeys, static_cast<long long>(a.Hkv) << a.page_shift),
                a.status, 633))
      return false;
    if (lane == 0) {
      const uint32_t dst = ring + stage * C::kStageBytes;
      mbar_arrive_expect_tx(bar0 + 8 * stage, C::kStageBytes);
      tma_load_3d(dst, &tm_k, bar0 + 8 * stage, 0, y, pid);
      tma_load_3d(dst + C::kTileBytes, &tm_v, bar0 + 8 * stage, 0, y, pid);
    }
    __syncwarp();
    return true;
  };

  // A sparse call asks for its first tiles before its first queries, the unit
  // looked up with them (a search less: 0.8 us of 25); a dense one fetches the
  // queries first (0.9 us of 100 the other way).
  Unit first{};
  if (!SPARSE && n_tiles > 0) {
    first = sched.unit_of(j0);
    fetch_q(first, 0);
  }
  Unit at_lane{};
  Tile cur = look_up(0, at_lane), next = cur;
  int pending = 0;                                  // stages with a copy in flight, one bit each
#pragma unroll
  for (int s = 0; s < C::kStages; ++s)
    if (s < n_tiles && issue(cur, s, s)) pending |= 1 << s;
  if (tid == 0) units[0] = SPARSE ? at_lane : first;
  if (SPARSE) fetch_q(shfl_unit(at_lane), 0);
  uint32_t phases = 0u;                             // parity of each stage's next completion
  bool ok = true;
  bool shared_unit = false;                         // thread 0: this CTA's last unit goes on
  // The tile that follows tile t in its stage; cur holds the tiles of `batch`.
  auto refill = [&](int t, int batch) {
    const int ahead = t + C::kStages, stage = t % C::kStages;
    if (ok && ahead < n_tiles && issue((ahead >> 5) == batch ? cur : next, ahead & 31, stage))
      pending |= 1 << stage;
  };
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (SPARSE) check.report(a.s, G * kThreads, a.page_shift, a.status);
  __syncthreads();

  int i = 0;                                        // tile of this warp
  for (int seg = 0; i < n_tiles; ++seg) {
    // ---- the CTA's part of one unit: pieces [j0 + i, j0 + end)
    const Unit u = units[seg & 1];
    const int end = min(j1, u.c0 + u.pieces(SPARSE)) - j0;
    const bool starts = j0 + i == u.c0, ends = j0 + end >= u.c0 + u.chunks;
    const bool whole = starts && ends;
    const bool some = j0 + i < u.c0 + u.chunks;     // else no keys, and no part, are left for this CTA
    // A CTA shares at most two units: the one it starts inside (slot 0) and
    // the one that goes on after it (slot 1).
    const int slot = starts ? 1 : 0;
    if (end < n_tiles) {
      // the buffers' last readers are two barriers back
      Unit nu = u;
      sched.advance(nu);
      fetch_q(nu, (seg + 1) & 1);
      if (tid == 0) units[(seg + 1) & 1] = nu;
    }

    // Queries as fp16 A fragments: row r or r + 8, columns kVals * c ...
    // (a k step's four columns of a thread are consecutive in memory).
    uint32_t qa[kK][4];
    float cs[2];                                    // log2(e) * scale, the row's power of two in it
    int lim[2];                                     // keys the row sees
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int rr = u.rb * kRows + r + 8 * hh;
      const bool on = rr < u.n * a.group;
      const int token = on ? rr / a.group : 0;
      lim[hh] = on ? (a.causal ? max(0, min(u.len, u.pos0 + token + 1)) : u.len) : 0;
      uint32_t w[D / 8];
      const uint32_t qp = sbase + C::kQOff + (((seg & 1) * kRows + r + 8 * hh) * D + kVals * c) * 2;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        const uint4 x = ld_shared_v4(qp + 16 * q);
        w[4 * q] = x.x;
        w[4 * q + 1] = x.y;
        w[4 * q + 2] = x.z;
        w[4 * q + 3] = x.w;
      }
      uint32_t mx = 0u;                             // largest exponent field of the row
#pragma unroll
      for (int q = 0; q < D / 8; ++q) mx = max(mx, max((w[q] >> 7) & 0xffu, (w[q] >> 23) & 0xffu));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = max(-126, min(126, static_cast<int>(mx) - 127));
      // a row with an infinity becomes NaN, as its scores say, also if all are -inf
      const float down = mx == 0xffu ? __int_as_float(0x7fffffff) : exp2i(-e);
      cs[hh] = a.scale_log2 * exp2i(e);
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t x = w[2 * kk + q];
          qa[kk][2 * q + hh] = pack_f16x2(__uint_as_float(x << 16) * down,
                                          __uint_as_float(x & 0xffff0000u) * down);
        }
      }
    }

    float o[kTiles8][4];
#pragma unroll
    for (int t = 0; t < kTiles8; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[t][q] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (; i < end; ++i) {
      const int stage = i % C::kStages;
      const Tile t = shfl_tile(cur, i & 31);
      if (t.pid >= 0 && ok) {
        ok = wait_bar_warp(bar0 + 8 * stage, phases >> stage & 1u, wc, kWaitKvFull);
        if (ok) pending &= ~(1 << stage);
      }
      if (t.pid >= 0 && ok) {
        phases ^= 1u << stage;
        const uint32_t kt = ring + stage * C::kStageBytes, vt = kt + C::kTileBytes;
        // ---- S = Q K^T, 32 keys in four n8 tiles
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
          const int key = 8 * n + r;
          uint32_t w[D / 16];                       // the thread's kVals codes of this key
          if constexpr (D == 128) {
            const uint4 x = ld_shared_v4(kt + key * 128 + (((2 * c) ^ (key & 7)) << 4));
            const uint4 y = ld_shared_v4(kt + key * 128 + (((2 * c + 1) ^ (key & 7)) << 4));
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
          } else {
            const uint4 x = ld_shared_v4(kt + key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          }
#pragma unroll
          for (int kk = 0; kk < kK; ++kk) {
            uint32_t b0, b1;
            e4m3x4_to_f16x4(w[kk], b0, b1);
            mma_f16(s[n], qa[kk], b0, b1);
          }
        }
        // ---- exponents, mask, running maximum
        const float f0 = cs[0] * t.ks, f1 = cs[1] * t.ks;
        const float lv = static_cast<float>(scale_exp(t.vs));
        const bool edge = t.key0 + kTileKeys > min(lim[0], lim[1]);
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            s[n][q] = fmaf(s[n][q], f0, lv);
            s[n][2 + q] = fmaf(s[n][2 + q], f1, lv);
            if (edge) {
              const int key = t.key0 + 8 * n + 2 * c + q;
              if (key >= lim[0]) s[n][q] = -INFINITY;
              if (key >= lim[1]) s[n][2 + q] = -INFINITY;
            }
            x0 = fmaxf(x0, s[n][q]);
            x1 = fmaxf(x1, s[n][2 + q]);
          }
        }
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) - kLift;
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) - kLift;
        const bool up = x0 > m[0] || x1 > m[1];
        if (__any_sync(0xffffffffu, up)) {
          const float n0 = fmaxf(m[0], x0), n1 = fmaxf(m[1], x1);
          const float b0 = n0 == -INFINITY ? 1.f : ex2_approx(m[0] - n0);
          const float b1 = n1 == -INFINITY ? 1.f : ex2_approx(m[1] - n1);
          m[0] = n0;
          m[1] = n1;
          l[0] *= b0;
          l[1] *= b1;
#pragma unroll
          for (int q = 0; q < kTiles8; ++q) {
            o[q][0] *= b0;
            o[q][1] *= b0;
            o[q][2] *= b1;
            o[q][3] *= b1;
          }
        }
        const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
        float sum0 = 0.f, sum1 = 0.f;
        uint32_t pa[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float p0 = ex2_approx(s[n][0] - m0), p1 = ex2_approx(s[n][1] - m0);
          const float p2 = ex2_approx(s[n][2] - m1), p3 = ex2_approx(s[n][3] - m1);
          sum0 += p0 + p1;
          sum1 += p2 + p3;
          pa[n >> 1][2 * (n & 1)] = pack_f16x2(p0, p1);
          pa[n >> 1][2 * (n & 1) + 1] = pack_f16x2(p2, p3);
        }
        const float inv = ex2_approx(-lv);
        l[0] = fmaf(sum0, inv, l[0]);
        l[1] = fmaf(sum1, inv, l[1]);
        // ---- O += P V: the thread's columns of four keys per k step, bytes
        // paired by key
        const int left = u.len - t.key0;             // keys of the tile that exist
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          constexpr int kW = kTiles8 / 4;            // words: columns kTiles8 * r ...
          uint32_t w[4][kW];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int key = 16 * kk + 2 * c + (q & 1) + 8 * (q >> 1);
            if constexpr (D == 128) {
              const uint4 x = ld_shared_v4(vt + key * 128 + ((r ^ (key & 7)) << 4));
              w[q][0] = x.x; w[q][1] = x.y; w[q][2] = x.z; w[q][3] = x.w;
            } else {
              const uint2 x =
                  ld_shared_v2(vt + key * 64 + (((r >> 1) ^ ((key >> 1) & 3)) << 4) + 8 * (r & 1));
              w[q][0] = x.x; w[q][1] = x.y;
            }
            // Slots behind the sequence's end hold anything, NaN codes too.
            if (left < kTileKeys && key >= left) {
#pragma unroll
              for (int z = 0; z < kW; ++z) w[q][z] = 0u;
            }
          }
#pragma unroll
          for (int z = 0; z < kW; ++z) {
            const uint32_t e0 = __byte_perm(w[0][z], w[1][z], 0x5140);
            const uint32_t e1 = __byte_perm(w[0][z], w[1][z], 0x7362);
            const uint32_t g0 = __byte_perm(w[2][z], w[3][z], 0x5140);
            const uint32_t g1 = __byte_perm(w[2][z], w[3][z], 0x7362);
            uint32_t b0, b1, b2, b3, c0, c1, c2, c3;
            e4m3x4_to_f16x4(e0, b0, b1);
            e4m3x4_to_f16x4(e1, b2, b3);
            e4m3x4_to_f16x4(g0, c0, c1);
            e4m3x4_to_f16x4(g1, c2, c3);
            mma_f16(o[4 * z], pa[kk], b0, c0);
            mma_f16(o[4 * z + 1], pa[kk], b1, c1);
            mma_f16(o[4 * z + 2], pa[kk], b2, c2);
            mma_f16(o[4 * z + 3], pa[kk], b3, c3);
          }
        }
      }
      // ---- the stage's next tile (the unit's last one waits for the join)
      __syncwarp();
      if (i + 1 < end) refill(i, i >> 5);
      if ((i & 31) == 8 && (i | 31) + 1 < n_tiles) next = look_up((i >> 5) + 1, at_lane);
      if ((i & 31) == 31) cur = next;
    }

    asm volatile("cp.async.wait_group 0;" ::: "memory");   // the next unit's queries
    // ---- the warps' results, joined
    const int free_stage = (end - 1) % C::kStages;
    auto join = [&](int w) {
      return reinterpret_cast<float*>(smem + (w * C::kStages + free_stage) * C::kStageBytes);
    };
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
      l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
      if (c == 0) ml[warp * kRows + r + 8 * hh] = make_float2(m[hh], l[hh]);
      // Row r's columns kVals c + ..., 16 bytes at a time, the slots permuted
      // within 128 bytes so that eight neighbouring lanes meet eight banks.
      float* base = join(warp) + (r + 8 * hh) * D + kVals * c;
      const int key = (c + 4 * (r & 1)) & (kVals / 4 - 1);
      if (!dcheck(in_range(smem_u32(base), kVals * 4, sbase, sbase + C::kRingBytes) && free_stage >= 0, a.status, 634))
        continue;
#pragma unroll
      for (int q = 0; q < kVals / 4; ++q) {
        // columns kVals c + 4 q ..: the first half of them are n = 2 c, then n = 2 c + 1
        const int t0 = (4 * q) % kTiles8, n1 = 4 * q / kTiles8;
        *reinterpret_cast<float4*>(base + 4 * (q ^ key)) =
            make_float4(o[t0][2 * hh + n1], o[t0 + 1][2 * hh + n1], o[t0 + 2][2 * hh + n1],
                        o[t0 + 3][2 * hh + n1]);
      }
    }
    __syncthreads();
    if (some && !whole && tid < kRows) {
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * kRows + tid].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = ml[w * kRows + tid];
        if (x.x != -INFINITY) ll += x.y * ex2_approx(x.x - mm);
        else if (x.y != x.y) ll = x.y;               // a NaN row
      }
      if (dcheck(inside((2 * cta + slot) * kRows + tid, 1, kPartRows), a.status, 635))
        a.part_ml[(2 * cta + slot) * kRows + tid] = make_float2(mm, ll);
    }
    for (int f = tid; some && f < kRows * (D / 4); f += kThreads) {
      const int row = f / (D / 4), q4 = f % (D / 4);
      const int rr = u.rb * kRows + row;
      if (rr >= u.n * a.group) continue;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * kRows + row].x);
      const int cq = q4 / (kVals / 4);
      const int key = (cq + 4 * (row & 1)) & (kVals / 4 - 1);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = ml[w * kRows + row];
        const float b = x.x == -INFINITY ? (x.y != x.y ? x.y : 0.f) : ex2_approx(x.x - mm);
        const float4 v = *reinterpret_cast<const float4*>(
            join(w) + row * D + kVals * cq + 4 * ((q4 % (kVals / 4)) ^ key));
        ll = fmaf(x.y, b, ll);
        acc.x = fmaf(v.x, b, acc.x);
        acc.y = fmaf(v.y, b, acc.y);
        acc.z = fmaf(v.z, b, acc.z);
        acc.w = fmaf(v.w, b, acc.w);
      }
      if (whole) {
        const int token = rr / a.group;
        const long long at = (static_cast<long long>(u.r0 + token) * a.Hkv + u.head) * a.group +
                             (rr - token * a.group);
        if (!dcheck(inside(at, 1, static_cast<long long>(a.s.T) * a.Hkv * a.group), a.status, 636)) continue;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2*>(a.o + at * D + 4 * q4) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (q4 == 0) a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else if (dcheck(inside((2ll * cta + slot) * kRows + row, 1, kPartRows), a.status, 637)) {
        *reinterpret_cast<float4*>(a.part_o + ((2ll * cta + slot) * kRows + row) * D + 4 * q4) = acc;
      }
    }
    if (tid == 0 && starts && !ends) {
      // The first CTA of a shared unit says what is to be joined.
      a.rec[2 * cta] = make_int4(u.r0, u.n, u.rb, u.head);
      a.rec[2 * cta + 1] = make_int4(cta_of(W, G, u.c0 + u.chunks - 1), W, 0, 0);
      shared_unit = true;
    }
    __syncthreads();
    fence_proxy_async_smem();       // TMA writes where the join was
    refill(end - 1, end >> 5);
  }
  allow_child();
  if (tid == 0 && !shared_unit) a.rec[2 * cta] = make_int4(0, 0, 0, 0);
  if (tid == 0) report_abort(misc[0], a.status);
  // Copies in flight land before the CTA exits (only after a wait gave up).
  for (int s = 0; s < C::kStages; ++s)
    if (pending >> s & 1) mbar_wait_drain(bar0 + 8 * s, phases >> s & 1u);
}

template <int D, bool SPARSE>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                     cudaStream_t stream) {
  auto kern = decode_kernel<D, SPARSE>;
  const int smem = DecCfg<D>::kSmemFixed + (SPARSE ? 0 : (a.s.B + 1) * 4);
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  kern<<<a.grid, kThreads, smem, stream>>>(tk, tv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_cache_join(D, kRows, a, stream);
}

}  // namespace

cudaError_t launch_cache_decode(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.selected != nullptr)
    return d == 64 ? launch_t<64, true>(tk, tv, a, stream) : launch_t<128, true>(tk, tv, a, stream);
  return d == 64 ? launch_t<64, false>(tk, tv, a, stream) : launch_t<128, false>(tk, tv, a, stream);
}

}  // namespace fattn
