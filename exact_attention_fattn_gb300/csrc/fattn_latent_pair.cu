// Attention over the paged latent cache for more than 64 rows a sequence: pairs of
// CTAs on two SMs (cta_group::2) work on 128 rows, so that what bounds the kernel
// for 64 rows, shared memory's 128 bytes a cycle, is used for twice the rows.
//
//   S^T = K Q^T      M = 128 (each CTA its 64 keys of a 128-key tile), N = 128 rows
//     (each CTA stages 64 rows of Q)
//   O^T += V^T P^T   M = 256 (each CTA half of the latent's columns, 128 at a time),
//     N = 128 rows (each CTA stages 64 rows of P), all 128 keys
//
// A CTA needs its own keys' rows whole for the first product, and half of the columns
// of all keys for the second.  The columns of its own keys that it has no use for
// after the first product make room, in the same place, for the columns that it
// needs of the other CTA's keys (from L2): the second product then finds each key
// half's columns at one address in both CTAs, and a tile takes no more than 72 KB.
// P goes where its rows are staged: half of it to the other CTA's shared memory.
//
// Per 128 keys and CTA: 2190 cycles of MMA; shared memory is read 245 KB (K 74, Q 74, V
// 65, P 32) and written 122 KB, 2870 cycles.  Two CTAs with 64 rows each need 5100.
//
// Softmax: tensor memory gives lanes 0-63 a CTA's keys for rows 0-63, lanes 64-127 the
// same keys for rows 64-127.  Both CTAs keep the same reference of every row, so they
// vote on each tile: where any row of either has a score above its reference by more
// than 2^8 (the first tile of a unit always has), they exchange the rows' maxima and
// move the references alike.  While the votes travel the probabilities are computed
// with the references there are.  What goes to the other CTA are asynchronous stores
// that count on a barrier there: a release at cluster scope waits for all that the
// thread has stored (votes and P by plain remote stores and releases took 5500 cycles
// a tile, 2500 of them waiting for the votes).
//
// Measured: 2 pieces of 1024 tokens, 16 heads, before keys up to 8192: 420 us (64 rows a CTA:
// 570), 1187 TFLOP/s; 64 single tokens of 128 heads over 500 to 8000 keys 100 (123).  A tile
// takes 3800 cycles in the first, 1750 of them issue of the products.  When it took 467 us
// neither the products bound it (with a quarter of their columns 459) nor L2 (two pairs a
// cluster with one copy of the keys for both 512) nor the softmax (16 warps 477): a tile's
// slots are free only after its second product, and from there copies, scores, softmax and
// the way of P to the other CTA follow one another with two tiles in turn, which is all that
// fits beside Q.  Less code in that chain is what helped (waits that stand once, copies'
// loops rolled): the roles share the instruction caches.
//
// Work split and join as in fattn_latent_attn.cu, a pair in a CTA's place.
//
// Warps: 0-7 softmax and results, 8 tensor memory and (leader) MMA issue, 9 loads, 10
// loads of the other CTA's keys, 11 the walk over the share.
// TMEM: S at 64 (tile & 1), O^T at 128 + 128 block.
#include "fattn_latent.cuh"

namespace fattn {

namespace {

constexpr int kRank = kLatentPairRank;
constexpr int kKeys = kLatentPairKeys;   // of a tile, half of them a CTA's
constexpr int kHalfKeys = 64;
constexpr int kRows = kLatentPairRows;
constexpr int kThreads = 384;
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr int kOtherWarp = 10;
constexpr int kWalkWarp = 11;
constexpr int kSegs = 2;
constexpr int kSegReaders = kSoftmaxWarps + 3;

struct C {
  static constexpr int kChunks = kRank / 64 + 1;
  static constexpr int kPairs = kRank / 128;         // 128-column parts of a cached row
  static constexpr int kBlocks = kPairs / 2;         // of them a CTA's own
  static constexpr int kChunk = kHalfKeys * 128;     // 64 rows, 64 columns
  static constexpr int kQOff = 0;
  static constexpr int kQBytes = kChunks * kChunk;
  static constexpr int kPOff = kQBytes;              // [2 key halves][64 rows][64 keys]
  static constexpr int kRingOff = kPOff + 2 * kChunk;
  static constexpr int kPairTile = 2 * kChunk;
  static constexpr int kRing = 8;                    // pairs
  static constexpr int kRopeOff = kRingOff + kRing * kPairTile;
  static constexpr int kBarOff = kRopeOff + kChunk;
  static_assert(kRing >= 2 * kPairs && kRing % kPairs == 0, "ring");
  static constexpr int kValid = kRing / kPairs;      // tiles whose masks are kept
  // barriers; those with (l) count for both CTAs in the leader's shared memory
  enum : int {
    kFull = 0,                    // (l) pair slots
    kEmpty = kFull + kRing,
    kRopeFull = kEmpty + kRing,   // (l)
    kRopeEmpty,
    kOther,                       // the other CTA's keys, in this CTA
    kOtherBoth = kOther + 2,      // (l) in both
    kQFull = kOtherBoth + 2,      // (l)
    kQEmpty,
    kSFull,
    kMask = kSFull + 2,
    kVote = kMask + kValid,
    kProb = kVote + 2,            // this CTA's rows of P, of either CTA's keys
    kProbPeer = kProb + 2,        // (l) the other's
    kExchange = kProbPeer + 2,    // the other CTA's maxima or sums
    kSync = kExchange + 2,        // this CTA's softmax warps
    kPvDone,                      // the products with either CTA's keys
    kMmaDone = kPvDone + 2,
    kSegFull,
    kSegEmpty = kSegFull + kSegs,
    kNumBars = kSegEmpty + kSegs
  };
  // Whether softmax warp `warp` of CTA `cta` arrives on that CTA's kProb + h: a warp that does has
  // also rescaled its part of O.  The first product, h = 0, writes to both CTAs' O, so all
  // warps of both count; the leader's need not again for the second.
  static constexpr bool counts_on(int h, int cta, int warp) { return h == 0 || h == cta || warp == 0; }
  // Arrivals that a phase of barrier `i` of CTA `cta` takes.
  static constexpr int arrivals(int i, int cta) {
    if (i == kOtherBoth || i == kOtherBoth + 1) return 2;
    if (i == kProb || i == kProb + 1) {
      int n = 0;
      for (int w = 0; w < kSoftmaxWarps; ++w) n += counts_on(i - kProb, cta, w) ? 1 : 0;
      return n;
    }
    if (i == kVote || i == kVote + 1 || i == kSync) return kSoftmaxWarps;
    return i >= kSegEmpty ? kSegReaders : 1;
  }
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;   // tmem, abort, votes[2], masks[]
  static constexpr int kPeerVoteOff = kMiscOff + 16 + 4 * kValid;   // [2][8]
  static constexpr int kSegOff = (kPeerVoteOff + 64 + 15) / 16 * 16;
  static constexpr int kOwnOff = kSegOff + kSegs * 32;      // [2][kRows] float
  static constexpr int kPeerOff = kOwnOff + 2 * kRows * 4;  // [2][kRows] float
  static constexpr int kAlphaOff = kPeerOff + 2 * kRows * 4;
  static constexpr int kSmem = kAlphaOff + kRows * 4;
  static_assert(kSmem <= kSmemMax && kNumBars < kThreads, "shared memory");
  __device__ static constexpr uint32_t col_s(uint32_t buf) { return 64 * buf; }
  __device__ static constexpr uint32_t col_o(int block) { return 128 + 128 * block; }
};

__device__ __forceinline__ void mma2_lead(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// To the barrier at this place in both CTAs.
__device__ __forceinline__ void commit2_lead(uint32_t bar, uint32_t lead) {
  const uint16_t mask = 3;
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          bar),
      "h"(mask), "r"(lead)
      : "memory");
}
// Like st_async_v4, four bytes.
__device__ __forceinline__ void st_async_u32(uint32_t cluster_addr, uint32_t x, uint32_t cluster_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(cluster_addr), "r"(x),
               "r"(cluster_bar)
               : "memory");
}
// An 8 x 8 matrix of 16-bit elements, two a lane, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// wait_warp for what the other CTA has stored and this one loads: votes, maxima and sums.  The
// other waits acquire at the CTA's scope: what they order is this CTA's own, or read by the
// tensor core after copies and stores that count on the barrier themselves.  All at the
// cluster's: 422 us for two pieces of 1024 tokens, 16 heads, before keys up to 8192, so 417.
__device__ __noinline__ bool wait_on_pair(uint32_t bar, uint32_t parity, long long budget, volatile uint32_t* abort,
                                          unsigned int site) {
  bool ok = true;
  const long long t0 = clock64();
  while (!mbar_try_wait_cl(bar, parity)) {
    if (*abort) ok = false;
    else if (clock64() - t0 > budget) {
      *abort = site;
      ok = false;
    }
    if (!ok) break;
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, const Waits& w, unsigned int site) {
  return __all_sync(0xffffffffu, mbar_try_wait_cl(bar, parity)) || wait_on_pair(bar, parity, w.budget, w.abort, site);
}

__global__ void __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ LatentAttnArgs args) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::kBarOff + 8u * i; };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  auto seg_at = [&](uint32_t i) -> const Seg& {
    return *reinterpret_cast<const Seg*>(smem + C::kSegOff + 32u * (i % kSegs));
  };
  volatile uint32_t* peer_votes = reinterpret_cast<volatile uint32_t*>(smem + C::kPeerVoteOff);   // [2][8]
  float* own = reinterpret_cast<float*>(smem + C::kOwnOff);        // [2 key quarters][kRows]
  float* peers = reinterpret_cast<float*>(smem + C::kPeerOff);     // [exchange & 1][kRows]
  float* alphas = reinterpret_cast<float*>(smem + C::kAlphaOff);   // [kRows]
  // Sums of the rounded probabilities, in P's place when a unit's products are done: this CTA's
  // [2 key quarters][kRows], then the other's [kRows].
  float* own_r = reinterpret_cast<float*>(smem + C::kPOff);
  float* peer_r = own_r + 2 * kRows;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  const bool leader = rank == 0u;
  const int pair = blockIdx.x >> 1, share = pair / args.span, block = pair - share * args.span;
  const int G = args.shares, group_rows = args.span * kRows;
  if (!dcheck((sbase & 1023u) == 0u && C::kSmem <= static_cast<int>(dynamic_smem_bytes()) && share < G, args.status, 701))
    return;                               // in both CTAs alike

  const SeqCheck mine(args.s, tid);
  if (tid < C::kNumBars) {
    mbar_init(bar(tid), C::arrivals(tid, rank));
    fence_barrier_init();
  }
  if (tid >= C::kNumBars && tid < C::kNumBars + 4 + C::kValid) misc[tid - C::kNumBars] = 0u;
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  __syncthreads();
  cluster_sync_all();                     // the other CTA's barriers are there
  if (warp == kMmaWarp) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(&misc[0])), 512);
    tmem_relinquish_pair();
  }
  const Share sh = locate_share<kKeys, latent_unit_cost(kRows), kThreads>(args, mine, group_rows, G, share, reinterpret_cast<long long*>(own),
                                                 reinterpret_cast<uint32_t*>(smem + C::kSegOff));   // read before the first segment
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const Waits wc{args.wait_budget, misc + 1};
  auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  auto wait_seg = [&](uint32_t i) { return wait_warp(bar(C::kSegFull + i % kSegs), (i / kSegs) & 1, wc, kWaitSegment); };
  auto done_seg = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kSegEmpty + i % kSegs));
  };
  auto first_row = [&](const Seg& s) { return static_cast<long long>(s.rg) * group_rows + block * kRows; };
  auto rows_of = [&](const Seg& s) { return static_cast<long long>(s.n) * args.Hq; };

  if (warp < kSoftmaxWarps) {
    // ================================================================ softmax
    // A warp has 32 of this CTA's 64 keys and 32 of the 128 rows, a thread four keys of
    // eight rows.  Every wait ends, and a warp whose wait ran out leaves.
    const float c = args.scale_log2;
    const int quarter = warp & 3, cols = 32 * (warp >> 2);          // of 64 columns of S
    const int row_base = 64 * (quarter >> 1) + cols, key_base = 32 * (quarter & 1) + (lane >> 2);
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    auto row_at = [&](int i) { return row_base + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1); };
    auto row_transposed = [&](int o) { return row_base + 8 * o + (lane >> 2); };
    const uint32_t home = quarter >> 1;                             // the CTA that stages these rows of P
    const uint32_t p_dst = map_shared(sbase + C::kPOff + rank * C::kChunk, home);
    uint32_t tiles = 0, syncs = 0, exchanges = 0;
    auto sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kSync));
      return wait_warp(bar(C::kSync), syncs++ & 1, wc, kWaitDrain);
    };
    // The rows' combined numbers of this CTA's keys (in own[0], own[1]) to the other.
    auto exchange = [&](bool sums) -> bool {
      if (!sync()) return false;
      const int b = C::kExchange + (exchanges & 1);
      if (tid < kRows) {
        const float x = own[tid], y = own[kRows + tid];
        st_async_u32(map_shared(smem_u32(peers + (exchanges & 1) * kRows + tid), peer),
                     __float_as_uint(sums ? x + y : fmaxf(x, y)), map_shared(bar(b), peer));
        if (sums)
          st_async_u32(map_shared(smem_u32(peer_r + tid), peer), __float_as_uint(own_r[tid] + own_r[kRows + tid]),
                       map_shared(bar(b), peer));
      }
      if (tid == 0) mbar_arrive_expect_tx(bar(b), kRows * (sums ? 8 : 4));
      return wait_pair(bar(b), exchanges++ >> 1 & 1, wc, kWaitDrain);
    };
    for (uint32_t si = 0; wait_seg(si); ++si) {
      const Seg s = seg_at(si);
      done_seg(si);
      if (s.flags & Seg::kLast) break;
      const long long row0 = first_row(s), rows = rows_of(s);
      if (row0 >= rows) continue;
      const int live = static_cast<int>(min(static_cast<long long>(kRows), rows - row0));
      // Keys that a row sees; rows behind the block's last see all (nothing of theirs is
      // stored, and a row of S, P and O depends on its own query only).
      auto lim_of = [&](int row) {
        if (!args.causal || row >= live) return s.len;
        return max(0, min(s.len, s.len - s.n + static_cast<int>(static_cast<unsigned int>(row0 + row) / args.Hq) + 1));
      };
      // A block's rows are of 128 tokens at most, so that what a row sees beyond the first fits a byte.
      const int lim_min = lim_of(0);
      uint32_t lim_more[2] = {0u, 0u};
      auto lim = [&](int i) { return lim_min + static_cast<int>(lim_more[i >> 2] >> (8 * (i & 3)) & 255u); };
      float m[8], l[8];
      // Sums of the rounded probabilities, taken when P is on its way: of rows row_at(i), or, where
      // they have been transposed for the other CTA, two of row_transposed(i / 2).
      float r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lim_more[i >> 2] |= static_cast<uint32_t>(lim_of(min(row_at(i), live - 1)) - lim_min) << (8 * (i & 3));
        m[i] = -FLT_MAX;
        l[i] = r[i] = 0.f;
      }
      bool holes = false, ok = true;
      for (int j = s.a; j < s.e; ++j, ++tiles) {
        const int kv0 = j * kKeys, mine0 = kv0 + kHalfKeys * static_cast<int>(rank);
        const bool first = j == s.a;
        if (!(ok = wait_warp(bar(C::kSFull + (tiles & 1)), (tiles >> 1) & 1, wc, kWaitSFull))) break;
        tc_fence_after();
        uint32_t lo[16], hi[16];           // keys of lanes 0-15 and 16-31 of the quarter
        const uint32_t ts = tmem + lane_off + C::col_s(tiles & 1) + cols;
        tmem_ld_rows(ts, lo);
        tmem_ld_rows(ts + (16u << 16), hi);
        if (!(ok = wait_warp(bar(C::kMask + tiles % C::kValid), (tiles / C::kValid) & 1, wc, kWaitKvFull))) break;
        const uint32_t mask = misc[4 + tiles % C::kValid];
        tmem_ld_wait(lo);
        tmem_ld_wait(hi);
        const bool edge = mask != 15u || kv0 + kKeys > s.len;
        // keys 0, 8, 16, 24 beyond the thread's first
        auto score = [&](int i, int k) -> uint32_t& {
          return (k < 2 ? lo : hi)[4 * (i >> 1) + 2 * (k & 1) + (i & 1)];
        };
        if (edge) {
          uint32_t want = 0u;
#pragma unroll
          for (int g = 0; g < 4; ++g) want |= (kv0 + 32 * g < s.len ? 1u : 0u) << g;
          holes |= (want & ~mask) != 0u;
        }
        if (edge || kv0 + kKeys > lim_min) {
          const bool there = mask >> (2 * rank + (quarter & 1)) & 1u;     // the warp's 32 keys
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!there || mine0 + key_base + 8 * k >= lim(i)) score(i, k) = __float_as_uint(-INFINITY);
        }
        auto val = [&](int i, int k) { return __uint_as_float(score(i, k)); };
        auto top_of = [&](int i) { return fmaxf(fmaxf(val(i, 0), val(i, 1)), fmaxf(val(i, 2), val(i, 3))); };
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaf(top_of(i), c, -m[i]));
        // The vote; two barriers in turn, as a CTA may be one tile ahead.
        const uint32_t turn = tiles & 1;
        const bool over = __any_sync(0xffffffffu, first || edge || top > kTau);
        if (lane == 0) {
          st_async_u32(map_shared(smem_u32(const_cast<uint32_t*>(&peer_votes[8 * turn + warp])), peer), over ? 1u : 0u,
                       map_shared(bar(C::kVote + turn), peer));
          if (over) misc[2 + turn] = tiles + 1;
          if (warp == 0) mbar_arrive_expect_tx(bar(C::kVote + turn), 4 * kSoftmaxWarps);
          else mbar_arrive(bar(C::kVote + turn));
        }
        // Probabilities, bf16 pairs of neighbouring rows: eight rows o, eight keys k.
        uint32_t w[4][4];
        float part[8];                     // this tile's sums
        auto compute = [&]() {
#pragma unroll
          for (int o = 0; o < 4; ++o)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float p0 = ex2_approx(fmaf(val(2 * o, k), c, -m[2 * o]));
              const float p1 = ex2_approx(fmaf(val(2 * o + 1, k), c, -m[2 * o + 1]));
              w[o][k] = pack_bf16x2(p0, p1);
              part[2 * o] = k == 0 ? p0 : part[2 * o] + p0;
              part[2 * o + 1] = k == 0 ? p1 : part[2 * o + 1] + p1;
            }
        };
        // For the other CTA, transposed in registers: lane 4 r + q has keys 2 q, 2 q + 1 of row r of
        // each chunk of eight keys; the four lanes of a row then swap words, so that lane q
        // has all of chunk q.
        auto transpose = [&]() {
          const int q = lane & 3;
#pragma unroll
          for (int o = 0; o < 4; ++o) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = movmatrix_trans(w[o][k]);
            const uint32_t a0 = __shfl_xor_sync(0xffffffffu, q & 2 ? u[0] : u[2], 2);
            const uint32_t a1 = __shfl_xor_sync(0xffffffffu, q & 2 ? u[1] : u[3], 2);
            const uint32_t k0 = q & 2 ? u[2] : u[0], k1 = q & 2 ? u[3] : u[1];
            const uint32_t b0 = __shfl_xor_sync(0xffffffffu, q & 1 ? k0 : k1, 1);
            const uint32_t b1 = __shfl_xor_sync(0xffffffffu, q & 1 ? a0 : a1, 1);
            const uint32_t m0 = q & 1 ? k1 : k0, m1 = q & 1 ? a1 : a0;
            // of chunk q: word q is m0, q ^ 2 m1, q ^ 1 b0, q ^ 3 b1
            w[o][0] = q == 0 ? m0 : (q == 2 ? m1 : (q == 1 ? b0 : b1));
            w[o][1] = q == 1 ? m0 : (q == 3 ? m1 : (q == 0 ? b0 : b1));
            w[o][2] = q == 2 ? m0 : (q == 0 ? m1 : (q == 3 ? b0 : b1));
            w[o][3] = q == 3 ? m0 : (q == 1 ? m1 : (q == 2 ? b0 : b1));
          }
        };
        if (!first) {
          compute();
          if (home != rank) transpose();
        }
        if (!(ok = wait_pair(bar(C::kVote + turn), (tiles >> 1) & 1, wc, kWaitPFull))) break;
        const bool moved = misc[2 + turn] == tiles + 1 || __any_sync(0xffffffffu, peer_votes[8 * turn + (lane & 7)] != 0u);
        // This CTA's keys' place in P is free.
        if (!first && !(ok = wait_warp(bar(C::kPvDone + rank), (tiles - 1) & 1, wc, kWaitMmaDone))) break;
        if (moved) {
          // ---- in both CTAs: some row's reference may move
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float t = top_of(i) * c;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
            if (lane < 4) own[(quarter & 1) * kRows + row_at(i)] = t;
          }
          if (!(ok = exchange(false))) break;
          const float* other = peers + ((exchanges - 1) & 1) * kRows;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = row_at(i);
            const float t = fmaxf(fmaxf(own[row], own[kRows + row]), other[row]);
            const bool move = t > m[i] + kTau;
            const float al = move ? ex2_approx(m[i] - t) : 1.f;
            if (move) m[i] = t;
            l[i] *= al;
            if (home == rank) r[i] *= al;
            if ((quarter & 1) == 0 && lane < 4) alphas[row] = al;
          }
          if (!(ok = sync())) break;
          if (home != rank) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] *= alphas[row_transposed(i >> 1)];
          }
          if (!first) {
            if (!(ok = wait_warp(bar(C::kPvDone + peer), (tiles - 1) & 1, wc, kWaitMmaDone))) break;
            tc_fence_after();
#pragma unroll 1
            for (int p = 0; p < C::kBlocks * 4; ++p) {
              uint32_t o[16];
              const int r0 = 64 * (warp >> 2) + 16 * (p & 3);
              const uint32_t at = tmem + lane_off + C::col_o(p >> 2) + r0;
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
          compute();
          if (home != rank) transpose();
          if (edge) {
            // Slots behind the end and pages that do not exist hold anything, and zero times a
            // NaN is a NaN.
            if (!(ok = wait_warp(bar(C::kOther + turn), (tiles >> 1) & 1, wc, kWaitKvFull))) break;
#pragma unroll 1
            for (int id = tid; id < 2 * C::kBlocks * 2 * kHalfKeys * 8; id += 32 * kSoftmaxWarps) {
              const int r = id >> 3 & (kHalfKeys - 1), half = id >> 9;      // half pairs, 64 rows of 8 pieces each
              const int h = half / (2 * C::kBlocks);                        // the keys' CTA
              if (kv0 + kHalfKeys * h + r < s.len && (mask >> (2 * h + (r >> 5)) & 1u)) continue;
              const uint32_t slot = (tiles * C::kPairs + (half >> 1)) % C::kRing;
              const uint32_t dst = sbase + C::kRingOff + slot * C::kPairTile + (half & 1) * C::kChunk + r * 128 + (id & 7) * 16;
              if (dcheck(in_range(dst, 16, sbase + C::kRingOff, sbase + C::kRopeOff), args.status, 704))
                st_shared_v4(dst, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            if (!(ok = sync())) break;
          }
        }
        // ---- P to where its rows are staged
        const int chunk = 4 * (quarter & 1);
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          if (home == rank) {
            const int row = cols + 8 * o + (lane & 7);
            const uint32_t dst = sbase + C::kPOff + rank * C::kChunk + row * 128 + (((chunk + (lane >> 3)) ^ (row & 7)) << 4);
            if (dcheck(in_range(dst, 16, sbase + C::kPOff, sbase + C::kRingOff), args.status, 702))
              stmatrix_x4_trans(dst, w[o][0], w[o][1], w[o][2], w[o][3]);
          } else {
            const int row = cols + 8 * o + (lane >> 2);
            const uint32_t off = row * 128 + (((chunk + (lane & 3)) ^ (row & 7)) << 4);
            if (dcheck(off + 16 <= static_cast<uint32_t>(C::kChunk), args.status, 703))
              st_async_v4(p_dst + off, w[o][0], w[o][1], w[o][2], w[o][3], map_shared(bar(C::kProb + rank), home));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kProb + rank));
        if (warp == 0) {
          // What the other CTA stores of P.  Its stores of the last tile must be there before its
          // barrier is armed for this one's: the products of that tile told the other CTA (it
          // waits for both), but the leader only of the first.
          if (leader && tiles > 0 && !(ok = wait_warp(bar(C::kProb + peer), (tiles - 1) & 1, wc, kWaitPFull))) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(C::kProb + peer), C::kChunk);
        } else if (C::counts_on(peer, rank, warp) && lane == 0) {
          mbar_arrive(bar(C::kProb + peer));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) l[i] += part[i];
#pragma unroll
        for (int o = 0; o < 4; ++o)
#pragma unroll
          for (int k = 0; k < 4; ++k) add_bf16(r[2 * o], r[2 * o + 1], w[o][k]);
      }
      if (!ok) break;
      // ---- results: this CTA's half of the columns, for all rows
      if (!wait_warp(bar(C::kPvDone), (tiles - 1) & 1, wc, kWaitOFull) || !wait_warp(bar(C::kPvDone + 1), (tiles - 1) & 1, wc, kWaitOFull))
        break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        if (lane < 4) own[(quarter & 1) * kRows + row_at(i)] = l[i];
        if ((quarter & 1) == 0 && lane < 4) alphas[row_at(i)] = m[i];
      }
      if (home == rank) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) r[i] += __shfl_xor_sync(0xffffffffu, r[i], off);
          if (lane < 4) own_r[(quarter & 1) * kRows + row_at(i)] = r[i];
        }
      } else {
#pragma unroll
        for (int o = 0; o < 4; ++o) {
          float x = r[2 * o] + r[2 * o + 1];
#pragma unroll
          for (int off = 1; off < 4; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
          if ((lane & 3) == 0) own_r[(quarter & 1) * kRows + row_transposed(o)] = x;
        }
      }
      if (!exchange(true)) break;
      tc_fence_after();
      const bool whole = s.whole();
      const long long slot = 2ll * pair + (s.flags & Seg::kStarts);
      const long long out0 = static_cast<long long>(s.r0) * args.Hq + row0;
      if (tid < kRows) {
        const float here = own[tid] + own[kRows + tid], there = peers[((exchanges - 1) & 1) * kRows + tid];
        const float here_r = own_r[tid] + own_r[kRows + tid], there_r = peer_r[tid];
        float lt = leader ? here + there : there + here;
        const float rt = leader ? here_r + there_r : there_r + here_r, mt = alphas[tid];
        // All scores of keys that the row sees are -inf: its query holds an infinity.
        if (lt == 0.f && !holes && lim_of(tid) > s.a * kKeys) lt = __int_as_float(0x7fffffff);
        if (leader && tid < live) {
          if (whole) args.lse[out0 + tid] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
          else args.part_ml[slot * kRows + tid] = make_float2(mt, lt);
        }
        alphas[tid] = row_factor(lt, rt, whole);
      }
      if (!sync()) break;
      const int col_base = kRank / 2 * static_cast<int>(rank) + 32 * quarter;     // of O
      if (whole) {
        // As in the kernel for 64 rows, through P's place: the other CTA writes to it again only
        // after the next unit's first exchange.
        const uint32_t stage = sbase + C::kPOff + warp * 2048;
#pragma unroll 1
        for (int t = 0; t < 2 * C::kBlocks; ++t) {
          const int r0 = 64 * (warp >> 2) + 32 * (t & 1);
          if (r0 >= live) continue;
          uint32_t lo[16], hi[16];
          const uint32_t at = tmem + lane_off + C::col_o(t >> 1) + r0;
          tmem_ld_rows(at, lo);
          tmem_ld_rows(at + (16u << 16), hi);
          tmem_ld_wait(lo);
          tmem_ld_wait(hi);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
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
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2), chunk = lane & 3;
            const uint4 w = ld_shared_v4(stage + row * 64 + ((chunk ^ (row >> 1 & 3)) << 4));
            if (r0 + row < live &&
                dcheck(inside(out0 + r0 + row, 1, static_cast<long long>(args.s.T) * args.Hq), args.status, 705))
              *reinterpret_cast<uint4*>(args.o + (out0 + r0 + row) * kRank + col_base + 128 * (t >> 1) + 8 * chunk) = w;
          }
        }
      } else {
#pragma unroll 1
        for (int p = 0; p < C::kBlocks * 4; ++p) {
          const int r0 = 64 * (warp >> 2) + 16 * (p & 3);
          if (r0 >= live) continue;
          uint32_t o[16];
          tmem_ld16(tmem + lane_off + C::col_o(p >> 2) + r0, o);
          float* to = args.part_o + (slot * kRows + r0) * kRank + col_base + 128 * (p >> 2) + lane;
          float f[16];
#pragma unroll
          for (int z = 0; z < 16; z += 4) *reinterpret_cast<float4*>(f + z) = *reinterpret_cast<const float4*>(alphas + r0 + z);
          tmem_ld_wait(o);
#pragma unroll
          for (int z = 0; z < 16; ++z)
            if (r0 + z < live && dcheck(slot < 2ll * (kSms / 2), args.status, 706)) to[z * kRank] = __uint_as_float(o[z]) * f[z];
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ================================================================ MMA issue
    const uint32_t lead = elect_lane();
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kRows, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(256, kRows, true, false);
    uint32_t tiles = 0, pvs = 0, q_count = 0;
    uint32_t ks = 0, kph = 0, vs = 0;   // slots and phases, as in the kernel for 64 rows
    auto ready = [&](int b, uint32_t parity) { return bar_done(bar(b), parity); };
    auto product4 = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
      const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, 16, 1024);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma2_lead(d, da + 2 * k, db + 2 * k, idesc_s, k > 0 ? 1u : acc, lead);
    };
    // The product with CTA h's keys of tile pvs.
    auto prob_there = [&](int h) { return ready(C::kProb + h, pvs & 1) && ready(C::kProbPeer + h, pvs & 1); };
    auto values = [&](int h, uint32_t acc) -> bool {
      // (P is there, part of it by the other CTA's stores)
      if (!wait_warp(bar(C::kOtherBoth + (pvs & 1)), (pvs >> 1) & 1, wc, kWaitKvFull)) return false;
      fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t db = sdesc_sw128(sbase + C::kPOff + h * C::kChunk, 16, 1024);
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b) {
        const uint64_t da = sdesc_sw128(sbase + C::kRingOff + vs * C::kPairTile, C::kChunk, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma2_lead(tmem + C::col_o(b), da + ((k * 2048) >> 4), db + 2 * k, idesc_o, k > 0 ? 1u : acc, lead);
        commit2_lead(bar(C::kEmpty + vs), lead);
        vs = vs + 1 == C::kRing ? 0u : vs + 1;
      }
      commit2_lead(bar(C::kPvDone + h), lead);
      if (h == 1) ++pvs;
      return true;
    };
    auto run = [&](const int n) -> bool {
      if (!wait_warp(bar(C::kQFull), q_count++ & 1, wc, kWaitQFull)) return false;
      tc_fence_after();
      for (int i = 0; i <= n; ++i) {
        int due = i > 0 ? 0 : 2;          // next product with the values of tile i - 1
        if (i < n) {
          // Scores of tile i, a part at a time as they come: the rotated columns, then 128 latent
          // ones each.  While a part is not there, the values of the tile before go first
          // where their probabilities are: only after that product are a tile's slots free.
          const uint32_t d = tmem + C::col_s(tiles & 1);
#pragma unroll 1
          for (int p = -1; p < C::kPairs; ++p) {
            const int b = p < 0 ? C::kRopeFull : C::kFull + static_cast<int>(ks);
            for (long long t0 = 0; !ready(b, p < 0 ? tiles & 1 : kph);) {
              if (due < 2 && prob_there(due)) {
                if (!values(due, i > 1 || due > 0 ? 1u : 0u)) return false;
                ++due;
              }
              const long long now = clock64();
              if (t0 == 0) t0 = now;
              if (now - t0 > wc.budget && *wc.abort == 0u) *wc.abort = kWaitKvFull;
              if (!__all_sync(0xffffffffu, *wc.abort == 0u)) return false;
            }
            tc_fence_after();
            if (p < 0) {
              product4(d, sbase + C::kRopeOff, sbase + C::kQOff + 2 * C::kPairs * C::kChunk, 0u);
              commit2_lead(bar(C::kRopeEmpty), lead);
            } else {
              const uint32_t k = sbase + C::kRingOff + ks * C::kPairTile, q = sbase + C::kQOff + 2 * p * C::kChunk;
              product4(d, k, q, 1u);
              product4(d, k + C::kChunk, q + C::kChunk, 1u);
              if (++ks == C::kRing) {
                ks = 0;
                kph ^= 1u;
              }
            }
          }
          commit2_lead(bar(C::kSFull + (tiles & 1)), lead);
          if (i + 1 == n) commit2_lead(bar(C::kQEmpty), lead);
          ++tiles;
        }
        for (; due < 2; ++due) {
          if (!wait_warp(bar(C::kProb + due), pvs & 1, wc, kWaitPFull) ||
              !wait_warp(bar(C::kProbPeer + due), pvs & 1, wc, kWaitPFull) || !values(due, i > 1 || due > 0 ? 1u : 0u))
            return false;
        }
      }
      return true;
    };
    for (uint32_t si = 0; wait_seg(si); ++si) {
      const Seg& s = seg_at(si);
      const int flags = uniform(s.flags), n = uniform(s.e - s.a);
      const bool on = uniform(first_row(s) < rows_of(s) ? 1 : 0) != 0;
      done_seg(si);
      if (flags & Seg::kLast) break;
      if (!on) continue;
      if (leader) {
        if (!run(n)) break;
      } else {
        // This CTA's P, told to the leader.
        bool ok = true;
        for (int i = 0; i < 2 * n && (ok = wait_warp(bar(C::kProb + (i & 1)), pvs & 1, wc, kWaitPFull)); ++i) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(map_shared(bar(C::kProbPeer + (i & 1)), 0));
          pvs += i & 1;
        }
        if (!ok) break;
      }
    }
    // No product may still be running when either CTA's memory goes.
    if (leader) commit2_lead(bar(C::kMmaDone), lead);
    mbar_drain_cl(bar(C::kMmaDone), 0);
    __syncwarp();
  } else if (warp == kLoadWarp || warp == kOtherWarp) {
    // ================================================================ loads
    // A tile's pages of the CTA's own keys, or of the other's: one, or two of 32 tokens.  A page
    // that does not exist is read as page 0, so that both CTAs' copies always count the
    // same bytes; its scores are masked and its values zeroed.
    const int page = 1 << args.page_shift, box = min(page, kHalfKeys), boxes = kHalfKeys / box;
    const uint32_t half = warp == kLoadWarp ? rank : peer;
    uint32_t tiles = 0, q_count = 0, ps = 0, eph = 0, pairs = 0;
    bool ok = true;
    for (uint32_t si = 0; ok && wait_seg(si); ++si) {
      const Seg s = seg_at(si);
      done_seg(si);
      if (s.flags & Seg::kLast) break;
      const long long row0 = first_row(s);
      if (row0 >= rows_of(s)) continue;
      if (warp == kLoadWarp) {
        if (q_count > 0 && !wait_warp(bar(C::kQEmpty), (q_count - 1) & 1, wc, kWaitQFull)) break;
        ++q_count;
        if (leader) mbar_arrive_expect_tx_w(bar(C::kQFull), 2 * C::kQBytes);
        tma2_load_3d_w(sbase + C::kQOff, &tm_q, map_shared(bar(C::kQFull), 0), 0,
                       uniform(static_cast<int>(static_cast<long long>(s.r0) * args.Hq + row0) + 64 * static_cast<int>(rank)), 0);
      }
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
        // The page of the tile's 32 keys from 32 g on.
        auto page_at = [&](int g) { return __shfl_sync(0xffffffffu, cur, ((j * kKeys + 32 * g) >> args.page_shift) - base); };
        auto good = [&](int p) { return p >= 0 && p < args.pages; };
        int pid0 = page_at(2 * half), pid1 = page_at(2 * half + 1);
        const int row = (j * kKeys + kHalfKeys * static_cast<int>(half)) & (page - 1);
        if (warp == kLoadWarp) {
          uint32_t mask = 0u;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int p = page_at(g);
            if (good(p)) mask |= 1u << g;
            else if (leader && lane == 0 && j * kKeys + 32 * g < s.len) record_bad_index(args.status, kSitePage);
          }
          pid0 = good(pid0) ? pid0 : 0;
          pid1 = good(pid1) ? pid1 : 0;
          auto load64 = [&](uint32_t dst, uint32_t b, int col) {
            tma2_load_3d_w(dst, &tm_k, b, col, row, pid0);
            if (boxes == 2) tma2_load_3d_w(dst + 4096, &tm_k, b, col, row, pid1);
          };
          if (tiles > 0 && !wait_warp(bar(C::kRopeEmpty), (tiles - 1) & 1, wc, kWaitKvEmpty)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx_w(bar(C::kRopeFull), 2 * C::kChunk);
          load64(sbase + C::kRopeOff, map_shared(bar(C::kRopeFull), 0), kRank);
#pragma unroll 1
          for (int p = 0; p < C::kPairs; ++p) {
            if (pairs >= C::kRing && !wait_warp(bar(C::kEmpty + ps), eph ^ 1u, wc, kWaitKvEmpty)) {
              ok = false;
              break;
            }
            if (p == 0) {
              if (lane == 0) {
                misc[4 + tiles % C::kValid] = mask;
                mbar_arrive(bar(C::kMask + tiles % C::kValid));
              }
              __syncwarp();
            }
            const uint32_t dst = sbase + C::kRingOff + ps * C::kPairTile, b = map_shared(bar(C::kFull + ps), 0);
            if (leader) mbar_arrive_expect_tx_w(bar(C::kFull + ps), 2 * C::kPairTile);
            load64(dst, b, 128 * p);
            load64(dst + C::kChunk, b, 128 * p + 64);
            ++pairs;
            if (++ps == C::kRing) {
              ps = 0;
              eph ^= 1u;
            }
          }
          if (!ok) break;
          // The ring has two tiles, too few for the time that they take to come from DRAM, so that the
          // next one is on its way to L2 meanwhile (64 sequences of 500 to 8000 keys, 128
          // heads: 113 us without, 105 so, 107 two tiles ahead, 106 before this tile's own
          // copies).  Where other pairs read the same keys they are there already.
          if (args.span == 1 && j + 1 < last_tile) {
            const int key = (j + 1) * kKeys + kHalfKeys * static_cast<int>(half);
            auto page_ahead = [&](int k) {
              const int at = (k >> args.page_shift) - base;
              const int a = __shfl_sync(0xffffffffu, cur, at & 31), b = __shfl_sync(0xffffffffu, nxt, at & 31);
              return at < 32 ? a : b;
            };
            constexpr int kWidth = kRank + kLatentRope;
            auto fetch = [&](int p, int k) {
              if (good(p) && lane == 0)
                prefetch_l2(args.data + p * args.page_stride + (k & (page - 1)) * kWidth, box * kWidth * 2);
            };
            const int p0 = page_ahead(key), p1 = page_ahead(key + 32);
            fetch(p0, key);
            if (boxes == 2) fetch(p1, key + 32);
            __syncwarp();
          }
        } else {
          // The other's keys, this CTA's columns, in place of its own keys' other columns once the
          // scores are computed.
          pid0 = good(pid0) ? pid0 : 0;
          pid1 = good(pid1) ? pid1 : 0;
          const uint32_t b = bar(C::kOther + (tiles & 1));
          if (!wait_warp(bar(C::kSFull + (tiles & 1)), (tiles >> 1) & 1, wc, kWaitSFull)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx_w(b, C::kBlocks * C::kPairTile);
#pragma unroll
          for (int i = 0; i < 2 * C::kBlocks; ++i) {
            const uint32_t slot = (tiles * C::kPairs + half * C::kBlocks + (i >> 1)) % C::kRing;
            const uint32_t dst = sbase + C::kRingOff + slot * C::kPairTile + (i & 1) * C::kChunk;
            const int col = kRank / 2 * static_cast<int>(rank) + 64 * i;
            tma_load_3d_w(dst, &tm_k, b, col, row, pid0);
            if (boxes == 2) tma_load_3d_w(dst + 4096, &tm_k, b, col, row, pid1);
          }
          if (!wait_warp(b, (tiles >> 1) & 1, wc, kWaitKvFull)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_cluster_relaxed(map_shared(bar(C::kOtherBoth + (tiles & 1)), 0));
          __syncwarp();
        }
      }
    }
    __syncwarp();
  } else if (warp == kWalkWarp) {
    // ================================================================ schedule
    const uint32_t* place = reinterpret_cast<const uint32_t*>(smem + C::kSegOff);
    Walker<kKeys, latent_unit_cost(kRows)> walk(args, group_rows, static_cast<int>(place[0]), static_cast<int>(place[1]), sh.j1 - sh.j0);
    __syncwarp();
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
      if (i >= kSegs && !wait_warp(bar(C::kSegEmpty + i % kSegs), (i / kSegs - 1) & 1, wc, kWaitSegment)) {
        any = false;
        break;
      }
      if (lane == 0) {
        const_cast<Seg&>(seg_at(i)) = x;
        mbar_arrive(bar(C::kSegFull + i % kSegs));
      }
      __syncwarp();
      if (!more) break;
    }
    if (lane == 0 && block == 0 && leader) {
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
  // Every copy must have landed before the pair ends.  In good order the products waited
  // for all of them; where a wait ran out they are given half a millisecond, hundreds
  // of times what a copy takes (a CTA cannot wait for those that the other counts).
  if (*wc.abort != 0u)
    for (const long long t0 = clock64(); clock64() - t0 < (1 << 20);) {
    }
  cluster_sync_all();                     // neither CTA's memory is used any more
  allow_child();
  if (tid == 0) report_abort(misc[1], args.status);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_latent_pair(const CUtensorMap& tk, const CUtensorMap& tq, const LatentAttnArgs& a, cudaStream_t stream) {
  auto kern = pair_kernel;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = 2 * a.span * a.shares;
  cfg.blockDim = kThreads;
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, tk, tq, a)) != cudaSuccess) return e;
  if (a.shares == 1) return cudaSuccess;   // nothing is shared
  return launch_latent_join_pairs(a, stream);
}

}  // namespace fattn
