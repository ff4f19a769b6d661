// Attention over the paged latent cache: one row of rank + 64 columns a token is
// its key for every query head, and the row's first rank columns are its value
// (the absorbed form: queries come multiplied with the keys' up-projection, and
// what is returned is still to be multiplied with the values').
//
//   S^T = K Q^T      [64 keys x N rows], rank + 64 columns summed
//   O^T += V^T P^T   [rank x N rows], 128 columns of V at a time
//
// Rows are N = 16, 32 or 64 (token, head) pairs of a sequence, and they are the
// products' N, not their M: with M = 128 rows the accumulator of 512 columns would
// fill tensor memory, and so would Q, 147 KB, shared memory; with 64 rows as M
// tcgen05 runs at half its rate.  So keys (64) are the first product's M and V's
// columns (128) the second's, and both read the same tile of the cache, K-major as
// K and MN-major as V^T.  A tile stays in shared memory between the two.  P^T goes
// through shared memory, K-major (stmatrix, transposed).
//
// Softmax: tensor memory gives a warp 16 keys of all rows (M = 64 uses 16 lanes of
// each quarter), so a thread has two keys of N / 4 rows, whose references m
// and sums l it keeps in registers.  A row's reference moves only when a score
// passes it by more than 2^8; whether one does is one vote of the warps, so
// that most tiles need no maximum over keys at all.  P is rounded to bf16 (half a
// step: 2^-8 of a probability), as V is, and O divided by the sum r of what the
// rounding leaves; scores, sums, references and accumulators are fp32.
//
// Work split: the key tiles of all units, in order, are dealt in equal contiguous
// shares; a unit is a group of `span` row blocks of one sequence, and a share is
// worked on by as many CTAs side by side, one a row block, so that the group's
// keys come out of DRAM once.  Units that shares split are joined in a second
// kernel, in order.
//
// Bound: the cache's bytes for 16 and 32 rows, shared memory for 64, whose 1920 cycles of
// products a 64-key tile (rank 512) are reads at 128 bytes a cycle, beside 576 for the
// tile's way in.  Measured, rank 512, one new token each: 64 sequences of 500 to 8000 keys, 16 heads
// 62 us (0.78 of the measured copy rate), 32 heads 68.6, 64 heads 78.7; 3 of 100000 to
// 131071, 32 heads 75.6 (0.79); one of 1000, 16 heads 12.0, of which the two launches, the
// schedule and the join are nearly all.  Products are issued in a fixed order by converged
// code: under branches that the compiler takes for divergent each took 82 cycles (when this
// kernel still had the calls of 128 heads, 64 sequences of them 178 us, then 152; copies
// under a lane's branch, 190 cycles each, 124.4, then 121.8).
//
// Warps: 0-3 softmax and results (0-7 with 64 rows, half of them each), then one for
// tensor memory and MMA issue, one for loads, one for the walk over the share (it
// publishes one segment after the other) and one for the loads of a tile's second page.
// TMEM: S at N (tile & 1), O^T at 2 N + N block.
#include "fattn_latent.cuh"

namespace fattn {

namespace {

constexpr int kKeys = kLatentKeys;
constexpr int kSegs = 4;
constexpr int kValid = 8;             // tiles whose masks are kept; more than the ring holds

template <int N, int R>
struct Cfg {
  // With 64 rows two warps share a quarter of tensor memory, 32 rows each.
  static constexpr int kHalves = N == 64 ? 2 : 1;
  static constexpr int kCols = N / kHalves;          // rows of a softmax warp
  static constexpr int kSoftmax = 128 * kHalves;     // threads
  static constexpr int kMmaWarp = 4 * kHalves;
  static constexpr int kLoadWarp = kMmaWarp + 1;
  static constexpr int kWalkWarp = kMmaWarp + 2;
  static constexpr int kLoad2Warp = kMmaWarp + 3;
  static constexpr int kThreads = 32 * (kMmaWarp + 4);
  static constexpr int kSegReaders = 4 * kHalves + 2;   // and one more for pages of 32 tokens
  static constexpr int kChunks = R / 64 + 1;         // 64-column parts of a query; the rotated one last
  static constexpr int kPairs = R / 128;             // 128-column parts of a cached row
  static constexpr int kQChunk = N * 128;
  static constexpr int kRopeTile = kKeys * 128;      // 64 columns of a tile
  static constexpr int kPairTile = 2 * kRopeTile;
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kChunks * kQChunk;
  static constexpr int kRingOff = kPOff + kQChunk;
  static constexpr int kMisc = 2304;
  static constexpr int kUnits = (kSmemMax - kRingOff - kMisc) / kRopeTile;
  // Two tiles at least: the scores of one are computed before the values of the
  // one before are done with.
#ifdef FATTN_LATENT_MIN_RING
  static constexpr int kRopes = 2;
  static constexpr int kRing = 2 * kPairs;
#else
  static constexpr int kRopes0 = (kUnits + 2 * kPairs) / (2 * kPairs + 1);
  static constexpr int kRopes = kRopes0 + ((kUnits - kRopes0) & 1);
  static constexpr int kRing = (kUnits - kRopes) / 2;
#endif
  static_assert(kRopes >= 2 && kRing >= 2 * kPairs && kRopes + 2 * kRing <= kUnits, "ring");
  static_assert(kRing / kPairs + 2 <= kValid, "masks");
  static constexpr int kRopeOff = kRingOff + kRing * kPairTile;
  static constexpr int kBarOff = kRopeOff + kRopes * kRopeTile;
  // pair_full[] pair_empty[] rope_full[] rope_empty[] q_full q_empty s_full[2] p_full
  // pv_done mma_done seg_full[] seg_empty[]
  static constexpr int kNumBars = 2 * kRing + 2 * kRopes + 7 + 2 * kSegs;
  // Arrivals that a phase of barrier `i` takes.  Where tiles have two pages, each of the two warps
  // that load arrives for its own, also for a page that is not there: neither may be a turn
  // of the ring behind the other, or it would wait for a phase that is over.
  static constexpr int arrivals(int i, bool two_pages) {
    const int rest = 2 * (kRing + kRopes);
    if (i < kRing || (i >= 2 * kRing && i < 2 * kRing + kRopes)) return two_pages ? 2 : 1;
    if (i == rest + 4) return kSoftmax;
    return i >= rest + 7 + kSegs ? kSegReaders + (two_pages ? 1 : 0) : 1;
  }
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;       // tmem, abort, start of the share
  static constexpr int kValidOff = kMiscOff + 32;
  static constexpr int kSegOff = (kValidOff + 4 * kValid + 15) / 16 * 16;
  static constexpr int kXOff = kSegOff + kSegs * 32;            // [4][N] float
  static constexpr int kAlphaOff = kXOff + 16 * N;              // [N] float
  static constexpr int kLimOff = kAlphaOff + 4 * N;             // [N] int
  static constexpr int kSmem = kLimOff + 4 * N;
  static_assert(kSmem <= kSmemMax && kNumBars < kThreads, "shared memory");
  __device__ static constexpr uint32_t col_s(uint32_t buf) { return N * buf; }
  __device__ static constexpr uint32_t col_o(int pair) { return 2 * N + N * pair; }
  static_assert(2 * N + N * kPairs <= 512, "tensor memory");
};

// Barrier of the softmax warps; true if `x` is in any thread.
template <int THREADS>
__device__ __forceinline__ bool barrier_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "n"(THREADS)
      : "memory");
  return r != 0;
}
template <int THREADS>
__device__ __forceinline__ void barrier_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// ------------------------------------------------------------------ kernel

template <int N, int R>
__global__ void __launch_bounds__(Cfg<N, R>::kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ LatentAttnArgs args) {
  using C = Cfg<N, R>;
  constexpr int kThreads = C::kThreads, kMmaWarp = C::kMmaWarp, kLoadWarp = C::kLoadWarp, kWalkWarp = C::kWalkWarp;
  constexpr int kLoad2Warp = C::kLoad2Warp;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBarOff;
  auto pair_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto pair_empty = [&](uint32_t s) { return bar0 + 8u * (C::kRing + s); };
  auto rope_full = [&](uint32_t s) { return bar0 + 8u * (2 * C::kRing + s); };
  auto rope_empty = [&](uint32_t s) { return bar0 + 8u * (2 * C::kRing + C::kRopes + s); };
  const uint32_t rest = bar0 + 16u * (C::kRing + C::kRopes);
  const uint32_t q_full = rest, q_empty = rest + 8u, p_full = rest + 32u, pv_done = rest + 40u, mma_done = rest + 48u;
  auto s_full = [&](uint32_t buf) { return rest + 16u + 8u * buf; };
  auto seg_full = [&](uint32_t i) { return rest + 56u + 8u * (i % kSegs); };
  auto seg_empty = [&](uint32_t i) { return rest + 56u + 8u * (kSegs + i % kSegs); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(smem + C::kValidOff);
  auto seg_at = [&](uint32_t i) -> const Seg& {
    return *reinterpret_cast<const Seg*>(smem + C::kSegOff + 32u * (i % kSegs));
  };
  float* xs = reinterpret_cast<float*>(smem + C::kXOff);          // [4][N]
  float* alphas = reinterpret_cast<float*>(smem + C::kAlphaOff);   // [N]
  int* lims = reinterpret_cast<int*>(smem + C::kLimOff);           // [N]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int share = blockIdx.x / args.span, block = blockIdx.x - share * args.span;
  const int G = args.shares, group_rows = args.span * N;
  if (!dcheck((sbase & 1023u) == 0u && C::kSmem <= static_cast<int>(dynamic_smem_bytes()) && share < G, args.status, 691))
    return;

  // The first sequence's numbers of each thread, on their way to the scan below.
  const SeqCheck mine(args.s, tid);
  if (tid < C::kNumBars) {
    mbar_init(bar0 + 8u * tid, C::arrivals(tid, args.page_shift == 5));
    fence_barrier_init();
  }
  if (tid == C::kNumBars) misc[1] = 0u;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&misc[0]), 512);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  // The scan's scratch is in the references' place, which nothing uses yet.
  const Share sh = locate_share<kKeys, latent_unit_cost(N), kThreads>(args, mine, group_rows, G, share, reinterpret_cast<long long*>(xs), misc + 4);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const Waits wc{args.wait_budget, reinterpret_cast<volatile uint32_t*>(&misc[1])};
  auto wait_seg = [&](uint32_t i) { return wait_warp(seg_full(i), (i / kSegs) & 1, wc, kWaitSegment); };
  auto done_seg = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty(i));
  };
  // First row of this CTA's block in the sequence's n * Hq (T * Hq < 2^31, and the
  // blocks' padding below 2^10).
  auto first_row = [&](const Seg& s) { return static_cast<long long>(s.rg) * group_rows + block * N; };
  auto rows_of = [&](const Seg& s) { return static_cast<long long>(s.n) * args.Hq; };

  // Every copy must have landed before the CTA exits.  Where a wait ran out, the two warps that
  // load may have asked for different tiles; then the copies are given half a
  // millisecond, hundreds of times what one takes.
  auto land = [&](uint32_t ropes, uint32_t pairs, uint32_t q_count) {
    const Waits drain{kDrainCycles, wc.abort};
    bool landed = true;
    for (uint32_t r = ropes > C::kRopes ? ropes - C::kRopes : 0; landed && r < ropes; ++r)
      landed = wait_warp(rope_full(r % C::kRopes), (r / C::kRopes) & 1, drain, kWaitDrain);
    for (uint32_t r = pairs > C::kRing ? pairs - C::kRing : 0; landed && r < pairs; ++r)
      landed = wait_warp(pair_full(r % C::kRing), (r / C::kRing) & 1, drain, kWaitDrain);
    if (landed && q_count > 0) landed = wait_warp(q_full, (q_count - 1) & 1, drain, kWaitDrain);
    if (!landed)
      for (const long long t0 = clock64(); clock64() - t0 < (1 << 20);) {
      }
    __syncwarp();
  };

  if (warp < kMmaWarp) {
    // ================================================================ softmax
    constexpr int NW = C::kCols, NC = NW / 4;   // rows of a warp; of a thread, two keys each
    auto softmax_any = [](bool x) { return barrier_any<C::kSoftmax>(x); };
    auto softmax_sync = [] { barrier_sync<C::kSoftmax>(); };
    const float c = args.scale_log2;
    const int quarter = warp & 3, col0 = NW * (warp >> 2);
    const int key_in = 16 * quarter + (lane >> 2);
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    auto col_of = [&](int i) { return col0 + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1); };
    uint32_t tiles = 0;                   // of this CTA so far: S and P V in turn
    // All decisions that a barrier follows are the same in these warps; a wait
    // that ran out makes the next vote end the loop for all.
    bool fail = false;
    for (uint32_t si = 0;; ++si) {
      fail |= !wait_seg(si);
      if (softmax_any(fail)) break;
      const Seg s = seg_at(si);
      done_seg(si);
      if (s.flags & Seg::kLast) break;
      const long long row0 = first_row(s), rows = rows_of(s);
      if (row0 >= rows) continue;
      const int live = static_cast<int>(min(static_cast<long long>(N), rows - row0));
      // Keys that a row sees.  Rows behind the block's last see all; nothing of theirs
      // is stored, and a row of S, P and O depends on its own query only.
      if (tid < N) {
        const int seen = s.len - s.n + static_cast<int>(static_cast<unsigned int>(row0 + tid) / args.Hq) + 1;
        lims[tid] = args.causal && tid < live ? max(0, min(s.len, seen)) : s.len;
      }
      softmax_sync();
      const int lim_min = lims[0];        // rows see no fewer keys than the first
      float m[NC], l[NC], r[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        m[i] = -FLT_MAX;
        l[i] = r[i] = 0.f;
      }
      bool holes = false;
      for (int j = s.a; j < s.e; ++j, ++tiles) {
        const int kv0 = j * kKeys;
        const uint32_t pair0 = tiles * C::kPairs;
        uint32_t x[NW / 2];
        fail |= !wait_warp(s_full(tiles & 1), (tiles >> 1) & 1, wc, kWaitSFull);
        // The masks came with the tile; its slots are not used again before P V.
        fail |= !wait_warp(pair_full(pair0 % C::kRing), (pair0 / C::kRing) & 1, wc, kWaitKvFull);
        tc_fence_after();
        tmem_ld_rows(tmem + lane_off + C::col_s(tiles & 1) + col0, x);
        const uint32_t mask = valid[tiles % kValid];
        tmem_ld_wait(x);
        const bool edge = mask != 3u || kv0 + kKeys > s.len;
        holes |= (((kv0 < s.len ? 1u : 0u) | (kv0 + 32 < s.len ? 2u : 0u)) & ~mask) != 0u;
        if (edge || kv0 + kKeys > lim_min) {
          const bool there0 = mask >> (key_in >> 5) & 1u, there1 = mask >> ((key_in + 8) >> 5) & 1u;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int lim = lims[col_of(i)] - kv0;
            uint32_t& x0 = x[4 * (i >> 1) + (i & 1)];
            uint32_t& x1 = x[4 * (i >> 1) + 2 + (i & 1)];
            if (!there0 || key_in >= lim) x0 = __float_as_uint(-INFINITY);
            if (!there1 || key_in + 8 >= lim) x1 = __float_as_uint(-INFINITY);
          }
        }
        auto s0 = [&](int i) { return __uint_as_float(x[4 * (i >> 1) + (i & 1)]); };
        auto s1 = [&](int i) { return __uint_as_float(x[4 * (i >> 1) + 2 + (i & 1)]); };
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NC; ++i) top = fmaxf(top, fmaf(fmaxf(s0(i), s1(i)), c, -m[i]));
        if (softmax_any(top > kTau || fail)) {
          // ---- some row's reference moves
          float mx[NC];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            mx[i] = fmaxf(s0(i), s1(i)) * c;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
            if (lane < 4) xs[quarter * N + col_of(i)] = mx[i];
          }
          if (j > s.a) fail |= !wait_warp(pv_done, (tiles - 1) & 1, wc, kWaitMmaDone);
          if (softmax_any(fail)) {
            fail = true;
            break;
          }
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int col = col_of(i);
            const float t = fmaxf(fmaxf(xs[col], xs[N + col]), fmaxf(xs[2 * N + col], xs[3 * N + col]));
            const bool move = t > m[i] + kTau;
            const float al = move ? ex2_approx(m[i] - t) : 1.f;
            if (move) m[i] = t;
            l[i] *= al;
            r[i] *= al;
            if (quarter == 0 && lane < 4) alphas[col] = al;
          }
          softmax_sync();
          if (j > s.a) {
            tc_fence_after();
#pragma unroll 1
            for (int p = 0; p < C::kPairs * NW / 16; ++p) {
              uint32_t o[16];
              const int r0 = col0 + 16 * p % NW;
              const uint32_t at = tmem + lane_off + C::col_o(16 * p / NW) + r0;
              tmem_ld16(at, o);
              const float4* al = reinterpret_cast<const float4*>(alphas + r0);
              tmem_ld_wait(o);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float4 f = al[z];
                o[4 * z] = __float_as_uint(__uint_as_float(o[4 * z]) * f.x);
                o[4 * z + 1] = __float_as_uint(__uint_as_float(o[4 * z + 1]) * f.y);
                o[4 * z + 2] = __float_as_uint(__uint_as_float(o[4 * z + 2]) * f.z);
                o[4 * z + 3] = __float_as_uint(__uint_as_float(o[4 * z + 3]) * f.w);
              }
              tmem_st16(at, o);
            }
            tmem_st_wait();
          }
        }
        // ---- probabilities, bf16 pairs of neighbouring rows
        uint32_t pk[NW / 4];
#pragma unroll
        for (int i = 0; i < NC; i += 2) {
          const float p00 = ex2_approx(fmaf(s0(i), c, -m[i])), p01 = ex2_approx(fmaf(s0(i + 1), c, -m[i + 1]));
          const float p10 = ex2_approx(fmaf(s1(i), c, -m[i])), p11 = ex2_approx(fmaf(s1(i + 1), c, -m[i + 1]));
          pk[i] = pack_bf16x2(p00, p01);
          pk[i + 1] = pack_bf16x2(p10, p11);
          l[i] += p00 + p10;
          l[i + 1] += p01 + p11;
        }
        if (tiles > 0) fail |= !wait_warp(pv_done, (tiles - 1) & 1, wc, kWaitMmaDone);   // P is free
#pragma unroll
        for (int i = 0; i < NW / 16; ++i) {
          const int row = col0 + 16 * i + 8 * (lane >> 4) + (lane & 7), chunk = 2 * quarter + (lane >> 3 & 1);
          const uint32_t dst = sbase + C::kPOff + row * 128 + ((chunk ^ (lane & 7)) << 4);
          if (dcheck(in_range(dst, 16, sbase + C::kPOff, sbase + C::kRingOff), args.status, 692))
            stmatrix_x4_trans(dst, pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
        if (edge) {
          // Slots behind the end and pages that were not loaded hold anything, and zero
          // times a NaN is a NaN.
#pragma unroll 1
          for (int id = tid; id < C::kPairs * 2 * kKeys * 8; id += C::kSoftmax) {
            const int r = id >> 3 & (kKeys - 1), half = id >> 9;   // 8 pieces a row, 64 rows a half pair
            if (kv0 + r < s.len && (mask >> (r >> 5) & 1u)) continue;
            const uint32_t slot = (pair0 + (half >> 1)) % C::kRing;
            const uint32_t dst = sbase + C::kRingOff + slot * C::kPairTile + (half & 1) * C::kRopeTile + r * 128 + (id & 7) * 16;
            if (dcheck(in_range(dst, 16, sbase + C::kRingOff, sbase + C::kRopeOff), args.status, 693))
              st_shared_v4(dst, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(p_full);
#pragma unroll
        for (int i = 0; i < NC; i += 2) {
          add_bf16(r[i], r[i + 1], pk[i]);
          add_bf16(r[i], r[i + 1], pk[i + 1]);
        }
      }
      // ---- results
      fail |= !wait_warp(pv_done, (tiles - 1) & 1, wc, kWaitOFull);
      float* rs = reinterpret_cast<float*>(smem + C::kPOff);   // [4][N]: no product reads P any more
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
          r[i] += __shfl_xor_sync(0xffffffffu, r[i], off);
        }
        const int col = col_of(i);
        if (lane < 4) {
          xs[quarter * N + col] = l[i];
          rs[quarter * N + col] = r[i];
        }
        if (quarter == 0 && lane < 4) alphas[col] = m[i];
      }
      if (softmax_any(fail)) break;
      tc_fence_after();
      const bool whole = s.whole();
      const long long slot = 2ll * blockIdx.x + (s.flags & Seg::kStarts);
      const long long out0 = static_cast<long long>(s.r0) * args.Hq + row0;
      if (tid < N) {
        float lt = (xs[tid] + xs[N + tid]) + (xs[2 * N + tid] + xs[3 * N + tid]);
        const float rt = (rs[tid] + rs[N + tid]) + (rs[2 * N + tid] + rs[3 * N + tid]), mt = alphas[tid];
        // All scores of keys that the row sees are -inf: its query holds an infinity.
        if (lt == 0.f && !holes && lims[tid] > s.a * kKeys) lt = __int_as_float(0x7fffffff);
        if (tid < live) {
          if (whole) args.lse[out0 + tid] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
          else args.part_ml[slot * N + tid] = make_float2(mt, lt);
        }
        alphas[tid] = row_factor(lt, rt, whole);
      }
      softmax_sync();
      if (whole) {
        // Rows of O^T, half of the block's a turn: pairs of rows to bf16, transposed through
        // this warp's part of P's place (32 columns a row, 16-byte chunks swizzled), so
        // that a store has 16 bytes a lane.
        constexpr int HB = NW / 2;
        const uint32_t stage = sbase + C::kPOff + warp * HB * 64;
#pragma unroll 1
        for (int t = 0; t < 2 * C::kPairs; ++t) {
          const int r0 = col0 + (t & 1) * HB;
          if (r0 >= live) continue;
          uint32_t lo[HB / 2], hi[HB / 2];          // columns 0 .. 15 and 16 .. 31 of the warp's
          const uint32_t at = tmem + lane_off + C::col_o(t >> 1) + r0;
          tmem_ld_rows(at, lo);
          tmem_ld_rows(at + (16u << 16), hi);
          tmem_ld_wait(lo);
          tmem_ld_wait(hi);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < HB / 8; ++i) {
            const float2 f = *reinterpret_cast<const float2*>(alphas + r0 + 8 * i + 2 * (lane & 3));
            auto pair_of = [&](const uint32_t* r) {
              return pack_bf16x2(__uint_as_float(r[0]) * f.x, __uint_as_float(r[1]) * f.y);
            };
            const int row = 8 * i + (lane & 7), chunk = lane >> 3;
            stmatrix_x4_trans(stage + row * 64 + ((chunk ^ (row >> 1 & 3)) << 4), pair_of(lo + 4 * i), pair_of(lo + 4 * i + 2),
                              pair_of(hi + 4 * i), pair_of(hi + 4 * i + 2));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < HB / 8; ++i) {
            const int row = 8 * i + (lane >> 2), chunk = lane & 3;
            const uint4 w = ld_shared_v4(stage + row * 64 + ((chunk ^ (row >> 1 & 3)) << 4));
            if (r0 + row < live &&
                dcheck(inside(out0 + r0 + row, 1, static_cast<long long>(args.s.T) * args.Hq), args.status, 694))
              *reinterpret_cast<uint4*>(args.o + (out0 + r0 + row) * R + 128 * (t >> 1) + 32 * quarter + 8 * chunk) = w;
          }
        }
      } else {
        // 16 rows at a time, a column a lane: whole lines.
#pragma unroll 1
        for (int p = 0; p < C::kPairs * NW / 16; ++p) {
          const int pair = 16 * p / NW, r0 = col0 + 16 * p % NW;
          if (r0 >= live) continue;
          uint32_t o[16];
          tmem_ld16(tmem + lane_off + C::col_o(pair) + r0, o);
          float* part = args.part_o + (slot * N + r0) * R + 128 * pair + 32 * quarter + lane;
          float f[16];
#pragma unroll
          for (int z = 0; z < 16; z += 4) *reinterpret_cast<float4*>(f + z) = *reinterpret_cast<const float4*>(alphas + r0 + z);
          tmem_ld_wait(o);
#pragma unroll
          for (int z = 0; z < 16; ++z)
            if (r0 + z < live && dcheck(slot < 2ll * kSms, args.status, 695)) part[z * R] = __uint_as_float(o[z]) * f[z];
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ================================================================ MMA issue
    const uint32_t lead = elect_lane();
    constexpr uint32_t idesc_s = idesc_bf16_f32(kKeys, N, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, N, true, false);
    uint32_t tiles = 0, pvs = 0, q_count = 0;
    // The bounds come through a shuffle, which tells the compiler that they are the
    // same in every lane.
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    auto product4 = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {   // 64 columns
      const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, 16, 1024);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_lead(d, da + 2 * k, db + 2 * k, idesc_s, k > 0 ? 1u : acc, lead);
    };
    auto keep_waiting = [&](long long& t0) -> bool {
      const long long now = clock64();
      if (t0 == 0) t0 = now;
      if (now - t0 > wc.budget && *wc.abort == 0u) *wc.abort = kWaitKvFull;
      return __all_sync(0xffffffffu, *wc.abort == 0u);
    };
    // Slots and phases of the tile whose scores come next, and of the one whose values do.
    uint32_t rs = 0, rph = 0, ks = 0, kph = 0, vs = 0;
    auto values = [&](uint32_t acc) {
      const uint64_t db = sdesc_sw128(sbase + C::kPOff, 16, 1024);
#pragma unroll 1
      for (int p = 0; p < C::kPairs; ++p) {
        const uint64_t da = sdesc_sw128(sbase + C::kRingOff + vs * C::kPairTile, C::kRopeTile, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_lead(tmem + C::col_o(p), da + ((k * 2048) >> 4), db + 2 * k, idesc_o, k > 0 ? 1u : acc, lead);
        commit_lead(pair_empty(vs), lead);
        vs = vs + 1 == C::kRing ? 0u : vs + 1;
      }
      commit_lead(pv_done, lead);
      ++pvs;
    };
    auto run = [&](const int n) -> bool {
      if (!wait_warp(q_full, q_count++ & 1, wc, kWaitQFull)) return false;
      tc_fence_after();
      for (int i = 0; i <= n; ++i) {
        bool due = i > 0;                 // values of tile i - 1
        if (i < n) {
          // Scores of tile i.  While its first columns are not there, the values of the tile
          // before go first where their probabilities are: a tile's slots are free only after
          // that product, and behind scores that wait it would hold up the loads.
          for (long long t0 = 0; !bar_done(rope_full(rs), rph) || !bar_done(pair_full(ks), kph);) {
            if (due && bar_done(p_full, pvs & 1)) {
              tc_fence_after();
              values(i > 1 ? 1u : 0u);
              due = false;
            }
            if (!keep_waiting(t0)) return false;
          }
          tc_fence_after();
          const uint32_t d = tmem + C::col_s(tiles & 1);
          product4(d, sbase + C::kRopeOff + rs * C::kRopeTile, sbase + C::kQOff + 2 * C::kPairs * C::kQChunk, 0u);
          commit_lead(rope_empty(rs), lead);
          if (++rs == C::kRopes) {
            rs = 0;
            rph ^= 1u;
          }
#pragma unroll
          for (int p = 0; p < C::kPairs; ++p) {
            if (p > 0 && !wait_warp(pair_full(ks), kph, wc, kWaitKvFull)) return false;
            const uint32_t k = sbase + C::kRingOff + ks * C::kPairTile, q = sbase + C::kQOff + 2 * p * C::kQChunk;
            product4(d, k, q, 1u);
            product4(d, k + C::kRopeTile, q + C::kQChunk, 1u);
            if (++ks == C::kRing) {
              ks = 0;
              kph ^= 1u;
            }
          }
          commit_lead(s_full(tiles & 1), lead);
          if (i + 1 == n) commit_lead(q_empty, lead);
          ++tiles;
        }
        if (due) {
          if (!wait_warp(p_full, pvs & 1, wc, kWaitPFull)) return false;
          tc_fence_after();
          values(i > 1 ? 1u : 0u);
        }
      }
      return true;
    };
    for (uint32_t si = 0; wait_seg(si); ++si) {
      const Seg& s = seg_at(si);
      const int flags = uniform(s.flags), n = uniform(s.e - s.a);
      const bool mine = uniform(first_row(s) < rows_of(s) ? 1 : 0) != 0;
      done_seg(si);
      if (flags & Seg::kLast) break;
      if (mine && !run(n)) break;
    }
    // No MMA may still be running when TMEM is released.
    commit_lead(mma_done, lead);
    mbar_wait_drain(mma_done, 0);
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ================================================================ TMA producer
    // Copies are issued by the converged warp, one lane of it elected by each: under a
    // branch on the lane their issue takes longer (190 cycles instead of 110), as
    // an MMA's does.  A block's queries are one copy; the cache's come 64 columns a copy (128 a
    // copy: two pieces of 1024 tokens, which pairs have now, 629 us, 64: 611).
    uint32_t tiles = 0, q_count = 0;
    uint32_t ropes = 0, pairs = 0;        // asked for so far
    uint32_t ps = 0, eph = 0;             // the next pair's slot, and the turn of the ring
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const int page = 1 << args.page_shift, box = min(page, kKeys), boxes = kKeys / box;
    bool ok = true;
    for (uint32_t si = 0; ok && wait_seg(si); ++si) {
      const Seg s = seg_at(si);
      done_seg(si);
      if (s.flags & Seg::kLast) break;
      const long long row0 = first_row(s);
      if (row0 >= rows_of(s)) continue;
      if (q_count > 0 && !wait_warp(q_empty, (q_count - 1) & 1, wc, kWaitQFull)) break;
      ++q_count;
      mbar_arrive_expect_tx_w(q_full, C::kChunks * C::kQChunk);
      const int q_row = uniform(static_cast<int>(static_cast<long long>(s.r0) * args.Hq + row0));
      tma_load_3d_w(sbase + C::kQOff, &tm_q, q_full, 0, q_row, 0);
      // 32 of the table's entries, one a lane, and the next 32 on their way.
      const int first_tile = uniform(s.a), last_tile = uniform(s.e);
      int base = (first_tile * kKeys) >> args.page_shift;
      int cur = page_of_lane(args, s.b, s.len, base), nxt = page_of_lane(args, s.b, s.len, base + 32);
      for (int j = first_tile; j < last_tile; ++j, ++tiles) {
        const int first = (j * kKeys) >> args.page_shift;
        if (first >= base + 32) {
          base += 32;
          cur = nxt;
          nxt = page_of_lane(args, s.b, s.len, base + 32);
        }
        auto page_at = [&](int p) { return __shfl_sync(0xffffffffu, cur, p - base); };
        // The tile's pages: one, or two of 32 tokens.
        int pid0 = page_at(first), pid1 = boxes == 2 ? page_at(first + 1) : -1;
        if (pid0 >= args.pages || pid1 >= args.pages || (pid0 < 0 && j * kKeys < s.len) ||
            (boxes == 2 && pid1 < 0 && j * kKeys + box < s.len)) {
          if (lane == 0) record_bad_index(args.status, kSitePage);
          if (pid0 >= args.pages) pid0 = -1;
          if (pid1 >= args.pages) pid1 = -1;
        }
        const uint32_t mask = (pid0 >= 0 ? (boxes == 1 ? 3u : 1u) : 0u) | (pid1 >= 0 ? 2u : 0u);
        const int row = (j * kKeys) & (page - 1);
        const uint32_t bytes = pid0 >= 0 ? static_cast<uint32_t>(box) * 128u : 0u;   // of this warp's page
        // A chunk of 64 columns, of the first page where there are two.
        auto load64 = [&](uint32_t dst, uint32_t bar, int chunk) {
          if (pid0 >= 0) tma_load_3d_w(dst, &tm_k, bar, 64 * chunk, row, pid0);
        };
        const uint32_t rs = tiles % C::kRopes;
        if (tiles >= C::kRopes && !wait_warp(rope_empty(rs), (tiles / C::kRopes - 1) & 1, wc, kWaitKvEmpty)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx_w(rope_full(rs), bytes);
        load64(sbase + C::kRopeOff + rs * C::kRopeTile, rope_full(rs), R / 64);
        ++ropes;
        if (lane == 0) valid[tiles % kValid] = mask;
        __syncwarp();
#pragma unroll 1
        for (int p = 0; p < C::kPairs; ++p) {
          if (pairs >= C::kRing && !wait_warp(pair_empty(ps), eph ^ 1u, wc, kWaitKvEmpty)) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + C::kRingOff + ps * C::kPairTile;
          mbar_arrive_expect_tx_w(pair_full(ps), 2 * bytes);
          load64(dst, pair_full(ps), 2 * p);
          load64(dst + C::kRopeTile, pair_full(ps), 2 * p + 1);
          ++pairs;
          if (++ps == C::kRing) {
            ps = 0;
            eph ^= 1u;
          }
        }
        if (!ok) break;
        // The next tile on its way to L2 in one piece, ahead of the boxes that wait for slots (64
        // sequences of 500 to 8000 keys, 16 heads 67.5 us without, 65.0 so, 66.1 two ahead,
        // 68.7 three).  With 64 rows it gains 2 % where a sequence has one block, but its code
        // costs 4 % where it has several (32 sequences of 4000 keys, 160 rows: 92 and 88).
        if constexpr (N < 64) {
          if (j + 1 < last_tile) {
            const int key = (j + 1) * kKeys;
            auto page_ahead = [&](int k) {
              const int at = (k >> args.page_shift) - base;
              const int a = __shfl_sync(0xffffffffu, cur, at & 31), b = __shfl_sync(0xffffffffu, nxt, at & 31);
              return at < 32 ? a : b;
            };
            constexpr int kWidth = R + kLatentRope;
            auto fetch = [&](int p, int k) {
              if (p >= 0 && p < args.pages && lane == 0)
                prefetch_l2(args.data + p * args.page_stride + (k & (page - 1)) * kWidth, box * kWidth * 2);
            };
            const int p0 = page_ahead(key), p1 = page_ahead(key + 32);
            fetch(p0, key);
            if (boxes == 2) fetch(p1, key + 32);
            __syncwarp();
          }
        }
      }
    }
    land(ropes, pairs, q_count);
  } else if (warp == kLoad2Warp && args.page_shift == 5) {
    // ================================================================ second pages
    // Where a tile has two pages (of 32 tokens) this warp loads the second one: 64 sequences of
    // 500 to 8000 keys, 64 heads 79.0 us, by one warp 84 (one role for both with its loads by
    // conditions 79.9, and 2 % slower for larger pages).
    uint32_t ropes = 0, pairs = 0, ps = 0, eph = 0;
    bool ok = true;
    for (uint32_t si = 0; ok && wait_seg(si); ++si) {
      const Seg s = seg_at(si);
      done_seg(si);
      if (s.flags & Seg::kLast) break;
      if (first_row(s) >= rows_of(s)) continue;
      int base = 2 * s.a;
      int cur = page_of_lane(args, s.b, s.len, base);
      for (int j = s.a; ok && j < s.e; ++j, ++ropes) {
        if (2 * j >= base + 32) cur = page_of_lane(args, s.b, s.len, base += 32);
        const int pid = __shfl_sync(0xffffffffu, cur, 2 * j + 1 - base);
        const bool there = pid >= 0 && pid < args.pages;
        const uint32_t rs = ropes % C::kRopes;
        if (ropes >= C::kRopes && !(ok = wait_warp(rope_empty(rs), (ropes / C::kRopes - 1) & 1, wc, kWaitKvEmpty))) break;
        const uint32_t bytes = there ? 4096u : 0u;
        mbar_arrive_expect_tx_w(rope_full(rs), bytes);
        if (there) tma_load_3d_w(sbase + C::kRopeOff + rs * C::kRopeTile + 4096, &tm_k, rope_full(rs), R, 0, pid);
#pragma unroll 1
        for (int p = 0; p < C::kPairs; ++p, ++pairs) {
          if (pairs >= C::kRing && !(ok = wait_warp(pair_empty(ps), eph ^ 1u, wc, kWaitKvEmpty))) break;
          const uint32_t dst = sbase + C::kRingOff + ps * C::kPairTile + 4096;
          mbar_arrive_expect_tx_w(pair_full(ps), 2 * bytes);
          if (there) {
            tma_load_3d_w(dst, &tm_k, pair_full(ps), 128 * p, 0, pid);
            tma_load_3d_w(dst + C::kRopeTile, &tm_k, pair_full(ps), 128 * p + 64, 0, pid);
          }
          if (++ps == C::kRing) {
            ps = 0;
            eph ^= 1u;
          }
        }
      }
    }
    land(ropes, pairs, 0);
  } else if (warp == kWalkWarp) {
    // ================================================================ schedule
    Walker<kKeys, latent_unit_cost(N)> walk(args, group_rows, static_cast<int>(misc[4]), static_cast<int>(misc[5]), sh.j1 - sh.j0);
    Seg s{};
    bool any = false;
    for (uint32_t i = 0;; ++i) {
      Seg x{};
      const bool more = walk.next(x);
      if (more) {
        s = x;
        any = true;
      } else {
        x.flags = Seg::kLast;
      }
      if (i >= kSegs && !wait_warp(seg_empty(i), (i / kSegs - 1) & 1, wc, kWaitSegment)) {
        any = false;
        break;
      }
      if (lane == 0) {
        const_cast<Seg&>(seg_at(i)) = x;
        mbar_arrive(seg_full(i));
      }
      __syncwarp();
      if (!more) break;
    }
    if (lane == 0 && block == 0) {
      // What is to be joined: the unit that this share starts and others go on with
      // (its last one).
      const bool shared_unit = any && (s.flags & (Seg::kStarts | Seg::kEnds)) == Seg::kStarts;
      args.rec[share] = shared_unit ? make_int4(s.r0, s.n, s.rg, cta_of(sh.W, sh.busy, sh.j1 - (s.e - s.a) + walk.nt - 1))
                                    : make_int4(0, 0, 0, 0);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  allow_child();
  if (tid == 0) report_abort(misc[1], args.status);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ join

struct Part {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void merge(Part& a, const Part& b) {
  const float m = fmaxf(a.m, b.m);
  const float x = ex2_approx(a.m - m), y = ex2_approx(b.m - m);
  a.m = m;
  a.l = fmaf(a.l, x, b.l * y);
  a.o.x = fmaf(a.o.x, x, b.o.x * y);
  a.o.y = fmaf(a.o.y, x, b.o.y * y);
  a.o.z = fmaf(a.o.z, x, b.o.z * y);
  a.o.w = fmaf(a.o.w, x, b.o.w * y);
}

// The rows of the units that shares start and others go on with.  Four groups of
// threads have 4 columns each of a row: a row or two of their own where a unit has few
// parts, a quarter of one row's parts where it has many.  A thread's four loads go out together:
// four parts of a row, or two of two rows for blocks of 128, whose units have few parts
// (whole calls: 64 sequences of 500 to 8000 keys, 128 heads 102.5 us with four of one, 101.2
// so; 8 of 4000, 64 rows a block, 28.5 and 30.4).  Every block counts the call's items and
// takes its own, so that there are no more blocks than work.
constexpr int kJoinGroups = 4;
constexpr int kJoinMany = 12;

template <int N, int R>
__global__ void __launch_bounds__(kJoinGroups * R / 4) join_kernel(const LatentAttnArgs a) {
  constexpr int kPer = N == kLatentPairRows ? 2 : 1, kAhead = 4 / kPer, kItem = kPer * kJoinGroups;
  __shared__ Part side[kJoinGroups][R / 4];
  __shared__ int4 recs[kSms];
  __shared__ int before[kSms + 1];
  const int G = a.shares, tid = threadIdx.x;
  wait_for_parent();
  auto first_of = [&](const int4& r) { return static_cast<long long>(r.z) * a.span * N; };   // of the sequence's rows
  auto rows_of = [&](const int4& r) {
    return static_cast<int>(min(static_cast<long long>(a.span * N), static_cast<long long>(r.y) * a.Hq - first_of(r)));
  };
  auto many = [&](int share, const int4& r) { return r.w - share + 1 > kJoinMany; };
  for (int t = tid; t < G; t += blockDim.x) {
    const int4 r = a.rec[t];
    recs[t] = r;
    before[t + 1] = r.y == 0 ? 0 : (many(t, r) ? rows_of(r) : (rows_of(r) + kItem - 1) / kItem);
  }
  if (tid == 0) before[0] = 0;
  __syncthreads();
  if (tid < 32) {                        // running sums, 32 shares at a time
    int sum = 0;
    for (int t0 = 0; t0 < G; t0 += 32) {
      int x = t0 + tid < G ? before[t0 + tid + 1] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (tid >= off) x += y;
      }
      if (t0 + tid < G) before[t0 + tid + 1] = sum + x;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const int q4 = tid % (R / 4), group = tid / (R / 4);
  for (int item = blockIdx.x; item < before[G]; item += gridDim.x) {
    int share = 0;
    for (int hi = G; hi - share > 1;) {
      const int mid = (share + hi) >> 1;
      if (before[mid] <= item) share = mid; else hi = mid;
    }
    const int4 rec = recs[share];
    const bool split = many(share, rec);
    const int rows = rows_of(rec), at_row = item - before[share];
    const int row0 = split ? at_row : kItem * at_row + group;
    Part p[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = Part{-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    // Behind the last part it is loaded again and not counted.
    const int step = split ? kJoinGroups : 1, ahead = split ? 4 : kAhead;
    auto part_of = [&](int t0, int i, int k) { return t0 + (split ? i * kAhead + k : k) * step; };
    auto row_of = [&](int i) { return split ? row0 : row0 + i * kJoinGroups; };
    for (int t0 = share + (split ? group : 0); t0 <= rec.w; t0 += ahead * step) {
      Part x[kPer][kAhead] = {};
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = row_of(i);
        if (row >= rows) continue;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int t = min(part_of(t0, i, k), rec.w);
          const long long at = (2ll * (t * a.span + row / N) + (t == share ? 1 : 0)) * N + row % N;
          if (!dcheck(inside(at, 1, 2ll * (N == kLatentPairRows ? kSms / 2 : kSms) * N), a.status, 696)) continue;
          const float2 ml = a.part_ml[at];
          x[i][k] = Part{ml.x, ml.y, reinterpret_cast<const float4*>(a.part_o + at * R)[q4]};
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (part_of(t0, i, k) <= rec.w) merge(p[i], x[i][k]);
    }
    if (split) {
      if constexpr (kPer > 1) merge(p[0], p[1]);
      side[group][q4] = p[0];
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int g = 1; g < kJoinGroups; ++g) merge(p[0], side[g][q4]);
      }
      __syncthreads();
      if (group != 0) continue;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int row = row_of(i);
      if ((split && i > 0) || row >= rows) continue;
      const long long out = static_cast<long long>(rec.x) * a.Hq + first_of(rec) + row;
      if (!dcheck(inside(out, 1, static_cast<long long>(a.s.T) * a.Hq), a.status, 697)) continue;
      const float inv = p[i].l == 0.f ? 0.f : 1.f / p[i].l;
      *reinterpret_cast<uint2*>(a.o + out * R + 4 * q4) =
          make_uint2(pack_bf16x2(p[i].o.x * inv, p[i].o.y * inv), pack_bf16x2(p[i].o.z * inv, p[i].o.w * inv));
      if (q4 == 0) a.lse[out] = p[i].l == 0.f ? -INFINITY : (p[i].m + log2f(p[i].l)) * kLn2;
    }
  }
}

template <int N, int R>
cudaError_t launch_join_t(const LatentAttnArgs& a, cudaStream_t stream) {
  const int rows = a.shares * a.span * N, most = kSms * 2048 / (kJoinGroups * R / 4);
  return launch_child(join_kernel<N, R>, rows < most ? rows : most, kJoinGroups * R / 4, 0, stream, a);
}

template <int N, int R>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tq, const LatentAttnArgs& a, cudaStream_t stream) {
  auto kern = latent_kernel<N, R>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), Cfg<N, R>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<a.span * a.shares, Cfg<N, R>::kThreads, Cfg<N, R>::kSmem, stream>>>(tk, tq, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.shares == 1) return cudaSuccess;   // nothing is shared
  return launch_join_t<N, R>(a, stream);
}

}  // namespace

cudaError_t launch_latent_join_pairs(const LatentAttnArgs& a, cudaStream_t stream) {
  return launch_join_t<kLatentPairRows, kLatentPairRank>(a, stream);
}

cudaError_t launch_latent_attn(int rows, int rank, const CUtensorMap& tk, const CUtensorMap& tq,
                               const LatentAttnArgs& a, cudaStream_t stream) {
  if (rank == 256)
    return rows == 16 ? launch_t<16, 256>(tk, tq, a, stream)
                      : (rows == 32 ? launch_t<32, 256>(tk, tq, a, stream) : launch_t<64, 256>(tk, tq, a, stream));
  return rows == 16 ? launch_t<16, 512>(tk, tq, a, stream)
                    : (rows == 32 ? launch_t<32, 512>(tk, tq, a, stream) : launch_t<64, 512>(tk, tq, a, stream));
}

}  // namespace fattn
