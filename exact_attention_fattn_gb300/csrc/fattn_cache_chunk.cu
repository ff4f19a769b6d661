// Attention over the paged 8-bit cache for many query rows per sequence
// (prompts, pieces of prompts, longer drafts).
//
// The rows of a unit are 256 (token, query head) pairs of one sequence that
// share a kv head, as two 128-row tiles; both meet every 128-key tile of the
// cache that one TMA load brings in.  With that many rows the products bound
// the call, 4 d operations per row and key, so they go to tcgen05:
//
//   S = Q K^T   on the codes themselves (kind::f8f6f4).  A bf16 query has 8
//     significant bits and an e4m3 code 4, so a row scaled by a power of two
//     is the sum of two e4m3 rows: hi = e4m3(x), lo = e4m3(x - hi), exact for
//     entries down to 2^-9 of the row's largest and off by at most 2^-10 of
//     224 below.  Two products at twice the 16-bit rate cost what one 16-bit
//     product would, and K needs no conversion.  A kernel in front splits Q
//     once and lays its rows out as the products read them.
//   O += P V    in fp16 (kind::f16): probabilities to fp16 in tensor memory
//     (one rounding, 2^-11), V's codes to fp16, exactly, by four converter
//     warps between the TMA ring and the MMA's tiles.  An e4m3 P would lose
//     2^-4 of every probability; splitting P as Q is would cost the softmax
//     warps three conversions per pair, and they set the pace already.
//
// Softmax with the page scales inside, as in the kernel for few rows: with
// c_p = scale log2(e) 2^e(row) kscale_p and l_p = log2 vscale_p,
//   x_j = c_p s_j + l_p,  P'_j = 2^(x_j - m),  l = sum_p 2^(-l_p) sum P'.
// A page is at least 32 tokens, so c and l_p are constant over each 32-column
// TMEM load and the row maximum comes from the load itself (tcgen05.ld.red).
// The reference moves only when a row's maximum passes it by more than 8, and P'
// is 2^7 times what it says, 2^15 at most: fp16 then holds probabilities down to
// 2^-31 of the largest.
//
// Bound: the chain of a row tile, its S (512 cycles of MMA), the softmax (about
// 1600), its P V (512) and the hand-overs, which the other tile's chain does not
// quite fill: 3370 cycles a step of both, 2048 of them MMA (2 x 2048 rows of 32
// heads on 16384 keys: 672 us, 1417 TFLOP/s, 0.73 of the measured bf16 rate,
// tensor pipe 60 % busy).  Handing P over in two parts, so that P V starts on the
// first, was slower (719 against 688 us).  Short prompts are bound by the units'
// ends: the softmax warps' set-up, masked tiles and stores.
//
// Work split: the key tiles of all units, in order, are dealt to the CTAs in
// equal contiguous shares, whatever the sequences' lengths and however many
// tiles causality cuts off; units that CTAs share are joined from partial
// results in a second kernel, in order.  A unit counts three tiles more than it
// has, about what its beginning and its end cost (5 rows of 8 heads on 32
// sequences: 80 us without them, 68.4 with three, 69.3 with five; 19 prompts of up
// to 895 tokens: 297 with three, 304 with five).
//
// Warps: 0-3 softmax of row tile 0, 4-7 of row tile 1, 8 tensor memory and MMA
// issue, 9 loads, 10 the walk over the CTA's share (it publishes one segment
// after the other in shared memory, so that no other role holds the schedule
// in registers), 11 idle, 12-15 conversion of V.  TMEM: S_t [128 t, 128 t + 128), P aliases S, O_t at 256 + d t.
#include <cuda_fp16.h>

#include <atomic>

#include "fattn_cache.cuh"

namespace fattn {

namespace {

#ifndef FATTN_CACHE_K_STAGES
#define FATTN_CACHE_K_STAGES 3
#endif
constexpr int kBM = 128;              // rows per tile
constexpr int kBN = 128;              // keys per tile
constexpr int kUnitRows = kChunkRows;
constexpr int kThreads = 512;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr int kWalkWarp = 10;
constexpr int kConvWarp0 = 12;
constexpr int kSegs = 4;              // segments in the shared ring
constexpr int kSegReaders = 8 + 2 + 4;   // warps that read each of them
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTau = 8.f;
constexpr float kLift = 7.f;
// Register split: 256 x 200 + 128 x 56 + 128 x 56 = 512 x 128, exactly the
// launch total, so setmaxnreg.inc can always complete.
constexpr int kLaunchRegs = 128;
constexpr int kSoftmaxRegs = 200;
constexpr int kCtrlRegs = 56;
constexpr int kConvRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kCtrlRegs + 128 * kConvRegs == kThreads * kLaunchRegs,
              "register split");
static_assert(kUnitRows == 2 * kBM, "rows of a unit");

template <int D>
struct ChunkCfg {
  static constexpr int kCodeTile = kBN * D;              // e4m3 tile: rows of D bytes, swizzled by D
  static constexpr int kQBytes = 2 * kCodeTile;          // hi, lo of one row tile
  static constexpr int kHalfTile = kBN * D * 2;          // fp16 V tile
  static constexpr int kHalfChunk = kBN * 128;           // 64 columns of it
  static constexpr int kKStages = FATTN_CACHE_K_STAGES;   // two at least
  static constexpr int kVStages = 2;                     // codes; two fp16 tiles follow
  static constexpr int kQOff = 0;
  static constexpr int kKOff = 2 * kQBytes;
  static constexpr int kVOff = kKOff + kKStages * kCodeTile;
  static constexpr int kHOff = kVOff + kVStages * kCodeTile;
  static constexpr int kBarOff = kHOff + 2 * kHalfTile;
  // k_full[] k_empty[] v_full[] v_empty[] h_full[2] h_empty[2] q_full[2]
  // s_full[2] p_full[2] o_full[2] o_empty[2] mma_done x_full x_empty
  // seg_full[] seg_empty[] q_empty[2]
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 17 + 2 * kSegs + 2;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;   // tmem, abort, valid[kVStages]
  static constexpr int kSegOff = (kMiscOff + 32 + 15) / 16 * 16;
  static constexpr int kXmlOff = kSegOff + kSegs * 64;      // [kBM] float2
  static constexpr int kPreOff = kXmlOff + kBM * 8;         // [B + 1] int
  static constexpr int kSmemFixed = kPreOff + 1024;
  __device__ static constexpr uint32_t col_s(int t) { return 128u * t; }
  __device__ static constexpr uint32_t col_o(int t) { return 256u + D * t; }
};

// Shared-memory matrix descriptor of an e4m3 tile: rows of D bytes, K-major,
// swizzled over D bytes (layout 2: 128 bytes, 4: 64 bytes), 8-row groups 8 D
// bytes apart.
template <int D>
__device__ __forceinline__ uint64_t sdesc_codes(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>((8 * D) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(D == 128 ? 2u : 4u) << 61;
  return d;
}

// Byte offset of 16-byte chunk c of row r of an e4m3 tile.
template <int D>
__device__ __forceinline__ uint32_t code_off(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// MMAs and their commits from one lane of the converged MMA warp, chosen once
// (`lead`) instead of in front of each.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_codes(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_halves(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// kind::f16 with fp16 A and B (format code 0), fp32 D; B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Key tiles that the rows [256 rb, 256 rb + rows) of a sequence need.  Row R
// sees pos0 + R / g + 1 keys, so rows before row E see at most pos0 + ceil(E / g).
// At least one, so that rows that see nothing are written, too.
__device__ __forceinline__ int tiles_of(const CacheAttnArgs& a, int n, int len, int rb, int rows) {
  int keys = len;
  if (a.causal) {
    const int end = min(n * a.group, rb * kUnitRows + rows);   // T * Hq < 2^31
    keys = len - n + (end + a.group - 1) / a.group;
  }
  return max(1, (keys + kBN - 1) / kBN);
}

// One CTA's part of a unit: key tiles [a, e) for the rows from 256 rb of a
// sequence.  Slot t (a softmax warpgroup with its TMEM columns) takes row tile
// t and key tiles from j0(t) up to last(t).  A unit of at most 128 rows is
// narrow: both slots take its one row tile, slot 0 the even key tiles of the
// part and slot 1 the odd ones, so that one slot's softmax runs beside the
// other's products there, too; slot 0's warps read both O's out of TMEM at the
// end.
struct __align__(16) Seg {
  int b, rb, head, nt;
  int r0, n, len, flags;
  int a, e, e0, pad;
  static constexpr int kStarts = 1, kEnds = 2, kNarrow = 4, kLast = 8;
  __device__ __forceinline__ bool narrow() const { return flags & kNarrow; }
  __device__ __forceinline__ bool whole() const { return (flags & 3) == 3; }
  __device__ __forceinline__ int j0(int t) const { return narrow() ? a + t : a; }
  __device__ __forceinline__ int last(int t) const { return t == 0 ? e0 : e; }
  __device__ __forceinline__ bool active(int t) const { return j0(t) < last(t); }
  // First row of the (sequence, head) in the split Q.
  __device__ __forceinline__ long long q_row(const CacheAttnArgs& a) const {
    return (static_cast<long long>(r0) * a.Hkv + static_cast<long long>(head) * n) * a.group;
  }
  // Row of the sequence's n * group of thread r of slot t (T * Hq < 2^31).
  __device__ __forceinline__ int row(int t, int r) const {
    return rb * kUnitRows + (narrow() ? 0 : t * kBM) + r;
  }
};
static_assert(sizeof(Seg) <= 64, "ring slot");

// Walks a CTA's share (one converged warp).
struct Walker {
  const CacheAttnArgs& a;
  const int* pre;           // pieces of work before each sequence
  long long left;           // pieces still to walk
  int b, rb, head, at, nt, nrb;   // at: piece of the unit, nt tiles and kChunkUnitCost more
  SeqInfo q;

  __device__ __forceinline__ void load_seq() {
    q = seq_info(a.s, b, a.page_shift);
    nrb = static_cast<int>((static_cast<long long>(q.n) * a.group + kUnitRows - 1) / kUnitRows);
  }
  __device__ __forceinline__ Walker(const CacheAttnArgs& args, const int* p, long long j0,
                                    long long j1)
      : a(args), pre(p), left(j1 - j0) {
    b = rb = head = at = nt = nrb = 0;
    if (left <= 0) return;
    int hi = a.s.B;         // the last b with pre[b] <= j0
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (pre[mid] <= j0) b = mid; else hi = mid;
    }
    load_seq();
    long long rem = j0 - pre[b];
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < nrb; base += 32) {
      const int i = base + lane;
      const long long w =
          i < nrb ? static_cast<long long>(tiles_of(a, q.n, q.len, i, kUnitRows) + kChunkUnitCost) * a.Hkv : 0;
      long long incl = w;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
      }
      const unsigned int past = __ballot_sync(0xffffffffu, incl > rem);
      if (past) {
        const int src = __ffs(past) - 1;
        rb = base + src;
        rem -= __shfl_sync(0xffffffffu, incl - w, src);
        break;
      }
      rem -= __shfl_sync(0xffffffffu, incl, 31);
    }
    nt = tiles_of(a, q.n, q.len, rb, kUnitRows);
    head = static_cast<int>(rem / (nt + kChunkUnitCost));
    at = static_cast<int>(rem - static_cast<long long>(head) * (nt + kChunkUnitCost));
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (at >= nt) {                     // pieces that stand for the unit itself
      left -= nt + kChunkUnitCost - at;
      at = 0;
      if (left <= 0) return false;
      if (++head == a.Hkv) {
        head = 0;
        if (++rb == nrb) {
          rb = 0;
          // work is left, so a sequence with rows follows
          do {
            if (++b >= a.s.B) return false;
            load_seq();
          } while (q.n == 0);
        }
        nt = tiles_of(a, q.n, q.len, rb, kUnitRows);
      }
    } else if (left <= 0) {
      return false;
    }
    s.b = b;
    s.rb = rb;
    s.head = head;
    s.r0 = q.r0;
    s.n = q.n;
    s.len = q.len;
    s.a = at;
    s.e = static_cast<int>(min(static_cast<long long>(nt), at + left));
    s.nt = nt;
    const bool narrow = static_cast<long long>(rb) * kUnitRows + kBM >= static_cast<long long>(q.n) * a.group;
    s.flags = (at == 0 ? Seg::kStarts : 0) | (s.e == nt ? Seg::kEnds : 0) | (narrow ? Seg::kNarrow : 0);
    s.e0 = narrow ? s.e : max(s.a, min(s.e, tiles_of(a, q.n, q.len, rb, kBM)));
    left -= s.e - s.a;
    at = s.e;
    return true;
  }
};

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {   // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// Page `first` + lane of a sequence, as the table has it; -1 past its end.
__device__ __forceinline__ int page_of_lane(const CacheAttnArgs& a, int b, int len, int first) {
  const int p = first + static_cast<int>(threadIdx.x & 31);
  if ((static_cast<long long>(p) << a.page_shift) >= len) return -1;
  return __ldg(a.s.table + static_cast<long long>(b) * a.s.max_pages + p);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ CacheAttnArgs args) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kBarOff;
  auto k_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto k_empty = [&](uint32_t s) { return bar0 + 8u * (C::kKStages + s); };
  auto v_full = [&](uint32_t s) { return bar0 + 8u * (2 * C::kKStages + s); };
  auto v_empty = [&](uint32_t s) { return bar0 + 8u * (2 * C::kKStages + C::kVStages + s); };
  const uint32_t rest = bar0 + 16u * (C::kKStages + C::kVStages);
  auto h_full = [&](uint32_t s) { return rest + 8u * s; };
  auto h_empty = [&](uint32_t s) { return rest + 16u + 8u * s; };
  auto q_full = [&](uint32_t t) { return rest + 32u + 8u * t; };
  auto s_full = [&](uint32_t t) { return rest + 48u + 8u * t; };
  auto p_full = [&](uint32_t t) { return rest + 64u + 8u * t; };
  auto o_full = [&](uint32_t t) { return rest + 80u + 8u * t; };
  auto o_empty = [&](uint32_t t) { return rest + 96u + 8u * t; };
  const uint32_t mma_done = rest + 112u, x_full = rest + 120u, x_empty = rest + 128u;
  auto seg_full = [&](uint32_t i) { return rest + 136u + 8u * (i % kSegs); };
  auto seg_empty = [&](uint32_t i) { return rest + 136u + 8u * (kSegs + i % kSegs); };
  auto q_empty = [&](uint32_t t) { return rest + 136u + 16u * kSegs + 8u * t; };
  const Seg* segs = reinterpret_cast<const Seg*>(smem + C::kSegOff);   // 64 bytes apart
  auto seg_at = [&](uint32_t i) -> const Seg& {
    return *reinterpret_cast<const Seg*>(reinterpret_cast<const uint8_t*>(segs) + 64u * (i % kSegs));
  };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile uint32_t* valid = misc + 2;   // per V stage: which 32-key groups were loaded
  int* pre = reinterpret_cast<int*>(smem + C::kPreOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, G = args.grid;
  [[maybe_unused]] constexpr long long kPartRows = part_rows(D, kUnitRows);
  [[maybe_unused]] const long long q_rows = static_cast<long long>(args.s.T) * args.Hkv * args.group;
  if (!dcheck(smem_u32(pre + args.s.B + 1) <= smem_u32(smem_raw) + dynamic_smem_bytes() &&
                  2ll * (cta + 1) * kUnitRows <= kPartRows && C::col_s(1) + kBN <= C::col_o(0) &&
                  C::col_o(1) + D <= 512,
              args.status, 641))
    return;

  if (tid == 0) {
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(h_full(t), 4);
      mbar_init(h_empty(t), 1);
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 128);
      mbar_init(o_full(t), 1);
      mbar_init(o_empty(t), 128);
    }
    mbar_init(mma_done, 1);
    mbar_init(x_full, 128);
    mbar_init(x_empty, 128);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(seg_full(i), 1);
      mbar_init(seg_empty(i), kSegReaders);
    }
    misc[1] = 0u;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&misc[0]), 512);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // ---- pieces of work before each sequence
  {
    __shared__ long long wtot[kThreads / 32];
    const int per = (args.s.B + kThreads - 1) / kThreads;
    const int b0 = min(args.s.B, tid * per), b1 = min(args.s.B, b0 + per);
    auto weight = [&](int b) -> long long {
      const SeqInfo q = seq_info(args.s, b, args.page_shift);
      if (!q.ok && cta == 0) record_bad_index(args.status, kSiteSeqStart);
      const int nrb = static_cast<int>((static_cast<long long>(q.n) * args.group + kUnitRows - 1) / kUnitRows);
      long long w = 0;
      for (int i = 0; i < nrb; ++i) w += tiles_of(args, q.n, q.len, i, kUnitRows) + kChunkUnitCost;
      return w * args.Hkv;
    };
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      pre[b] = static_cast<int>(sum);
      sum += weight(b);
    }
    long long incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += t;
    }
    if (lane == 31) wtot[warp] = incl;
    __syncthreads();
    long long at = incl - sum;
    for (int w = 0; w < warp; ++w) at += wtot[w];
    for (int b = b0; b < b1; ++b) pre[b] += static_cast<int>(at);
    if (tid == kThreads - 1) pre[args.s.B] = total_of(at + sum, args.status);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const Waits wc{args.wait_budget, reinterpret_cast<volatile uint32_t*>(&misc[1])};
  const long long W = pre[args.s.B];
  // Segment i of the CTA; a reader that is done with it hands it back.
  auto wait_seg = [&](uint32_t i) {
    return wait_bar_warp(seg_full(i), (i / kSegs) & 1, wc, kWaitSegment);
  };
  auto done_seg = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty(i));
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================================================================ softmax
    const int t = warp >> 2;              // row tile
    const int wq = warp & 3;
    const int r_tile = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    const int pages_log = 7 - args.page_shift;   // log2 of the pages per key tile
    uint32_t s_count = 0, o_count = 0, x_count = 0, o1_count = 0;   // o1: slot 1's, as slot 0 counts them
    float2* xml = reinterpret_cast<float2*>(smem + C::kXmlOff);
    bool ok = true;

    wait_for_parent();                    // q_scale
    for (uint32_t si = 0; ok; ++si) {
      if (!(ok = wait_seg(si))) break;
      const Seg& s = seg_at(si);
      if (s.flags & Seg::kLast) break;
      // Keys the row sees.  Rows past the unit's last see all, so that they need no
      // mask.  Their queries are whatever shared memory held, and so are their
      // scores, NaN included; but a row of S, P and O depends on its own query
      // only, a rescale that such a row sets off multiplies the others by 1, and
      // nothing of such a row is stored.
      int lim = s.len;
      float m_ref = -INFINITY, l = 0.f, c0 = 1.f;
      {
        const int rr = s.row(t, r_tile);
        if (rr < s.n * args.group && dcheck(inside(s.q_row(args) + rr, 1, q_rows), args.status, 642)) {
          if (args.causal) lim = max(0, min(s.len, s.len - s.n + rr / args.group + 1));
          // log2(e) * scale times the power of two taken out of the row
          c0 = args.scale_log2 * args.q_scale[s.q_row(args) + rr];
        }
      }
      const int jb = s.j0(t), nj = s.last(t), step = s.narrow() ? 2 : 1;
      // 32 pages, one per lane: page, K scale, log2 of the V scale
      int w_base = 0, w_pid = -1;
      float w_ks = 0.f, w_lv = 0.f;
      auto load_window = [&](int first) {
        w_base = first;
        w_pid = page_of_lane(args, s.b, s.len, first);
        if (w_pid >= args.pages) w_pid = -1;   // the loader reports it
        w_ks = w_lv = 0.f;
        if (w_pid >= 0) {
          const long long sc = static_cast<long long>(w_pid) * args.Hkv + s.head;
          w_ks = __ldg(args.k_scale + sc);
          w_lv = static_cast<float>(scale_exp(__ldg(args.v_scale + sc)));
        }
      };
      if (jb < nj) load_window(jb << pages_log);
      for (int j = jb; j < nj; j += step) {
        if (((j + 1) << pages_log) - w_base > 32) load_window(j << pages_log);
        // Per 32 columns: factor of the exponent (positive, so that a masked
        // score stays -inf; |S| < 2^26, so what is lost is far below the last
        // bit of a probability), log2 of the V scale, and keys to be seen.
        const int kv0 = j * kBN;
        const int p0 = (kv0 >> args.page_shift) - w_base;
        auto page_at = [&](int g) { return p0 + (32 * g >> args.page_shift); };
        auto cg_of = [&](int g) {
          return fmaxf(c0 * __shfl_sync(0xffffffffu, w_ks, page_at(g)), 1e-37f);
        };
        auto lg_of = [&](int g) { return __shfl_sync(0xffffffffu, w_lv, page_at(g)); };
        auto lim_of = [&](int g) {
          return __shfl_sync(0xffffffffu, w_pid, page_at(g)) < 0 ? 0 : lim - kv0 - 32 * g;
        };
        const unsigned int missing = __ballot_sync(0xffffffffu, w_pid < 0);
        const int p3 = page_at(3);
        const bool hole = (missing >> p0 & (0xffffffffu >> (31 - (p3 - p0)))) != 0u;
        const bool masked = __any_sync(0xffffffffu, kv0 + kBN > lim || hole);
        ok = wait_bar_warp(s_full(t), s_count & 1, wc, kWaitSFull);
        if (!ok) break;
        ++s_count;
        tc_fence_after();
        // ---- scores, each 32 columns with their maximum
        uint32_t s0[32], s1[32], s2[32], s3[32];
        float mg[4], cg[4], lg[4];
        tmem_ld32_max(tS + 0, s0, mg[0]);
        tmem_ld32_max(tS + 32, s1, mg[1]);
        tmem_ld32_max(tS + 64, s2, mg[2]);
        tmem_ld32_max(tS + 96, s3, mg[3]);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          cg[g] = cg_of(g);
          lg[g] = lg_of(g);
        }
        tmem_ld_wait32(s0);
        reg_fence32(s1);
        reg_fence32(s2);
        reg_fence32(s3);
#pragma unroll
        for (int g = 0; g < 4; ++g) reg_fence1(mg[g]);
        uint32_t* sv[4] = {s0, s1, s2, s3};
        if (masked) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int lh = lim_of(g);
            if (!__any_sync(0xffffffffu, lh < 32)) continue;   // most of a diagonal tile
            mg[g] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (i >= lh) sv[g][i] = __float_as_uint(-INFINITY);
              mg[g] = fmaxf(mg[g], __uint_as_float(sv[g][i]));
            }
          }
        }
        const float m_new = fmaxf(fmax3(fmaf(mg[0], cg[0], lg[0]), fmaf(mg[1], cg[1], lg[1]),
                                        fmaf(mg[2], cg[2], lg[2])),
                                  fmaf(mg[3], cg[3], lg[3]));
        const bool need = m_new > m_ref + kTau;
        const bool rescale = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (rescale) {
          alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
          if (need) m_ref = m_new;
          l *= alpha;
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref - kLift;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t pk[16];
          uint64_t e2 = 0ull;
          const uint64_t c2 = splat2(cg[g]), nm2 = splat2(lg[g] - m_use);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t x0, x1;
            unpack2(ffma2(pack2(sv[g][2 * i], sv[g][2 * i + 1]), c2, nm2), x0, x1);
            const float a0 = ex2_approx(__uint_as_float(x0));
            const float a1 = ex2_approx(__uint_as_float(x1));
            const __half2 h = __floats2half2_rn(a0, a1);
            pk[i] = *reinterpret_cast<const uint32_t*>(&h);
            e2 = fadd2(e2, pack2(__float_as_uint(a0), __float_as_uint(a1)));
          }
          tmem_st16(tS + 16 * g, pk);
          uint32_t u0, u1;
          unpack2(e2, u0, u1);
          l = fmaf(__uint_as_float(u0) + __uint_as_float(u1), ex2_approx(-lg[g]), l);
        }
        if (rescale && j > jb) {
          // P V of the last tile has completed: it was issued before this S.
          const uint64_t a2 = splat2(alpha);
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ch += 2) {
            uint32_t o0[32], o1[32];
            tmem_ld32(tO + 32 * ch, o0);
            tmem_ld32(tO + 32 * ch + 32, o1);
            tmem_ld_wait32(o0);
            reg_fence32(o1);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              unpack2(fmul2(pack2(o0[2 * i], o0[2 * i + 1]), a2), o0[2 * i], o0[2 * i + 1]);
              unpack2(fmul2(pack2(o1[2 * i], o1[2 * i + 1]), a2), o1[2 * i], o1[2 * i + 1]);
            }
            tmem_st32(tO + 32 * ch, o0);
            tmem_st32(tO + 32 * ch + 32, o1);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(t));
      }
      if (!ok) break;
      // ---- results
      const bool whole = s.whole();
      const int rr = s.row(t, r_tile);
      const long long slot = 2ll * cta + (s.flags & Seg::kStarts);
      const bool on = rr < s.n * args.group &&
                      dcheck(inside(slot * kUnitRows + t * kBM + r_tile, 1, kPartRows), args.status, 643);
      float4* part = reinterpret_cast<float4*>(args.part_o + (slot * kUnitRows + t * kBM + r_tile) * D);
      float2* part_ml = args.part_ml + slot * kUnitRows + t * kBM + r_tile;
      if (jb >= nj) {
        // Nothing for this row tile here (causality): an empty part.
        if (!s.narrow() && !whole && on) {
#pragma unroll 1
          for (int i = 0; i < D / 4; ++i) part[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          *part_ml = make_float2(-INFINITY, 0.f);
        }
        if (t == 0 && s.active(1)) ++o1_count;
        done_seg(si);
        continue;
      }
      // (Slot 0 waits for a narrow unit's second O; it is long there when slot 1
      // comes to its next one.)
      if (!(s.narrow() && t == 1))
        ok = wait_bar_warp(o_full(t), o_count & 1, wc, kWaitOFull);
      if (!ok) break;
      ++o_count;
      tc_fence_after();
      if (s.narrow() && t == 1) {
        if (x_count > 0) {
          ok = wait_bar_warp(x_empty, (x_count - 1) & 1, wc, kWaitDrain);
          if (!ok) break;
        }
        ++x_count;
        xml[r_tile] = make_float2(m_ref, l);
        mbar_arrive(x_full);
        done_seg(si);
        continue;
      }
      const bool joined = s.narrow() && s.e - s.a > 1;
      float a0 = 1.f, a1 = 0.f;
      if (joined) {
        ok = wait_bar_warp(x_full, x_count & 1, wc, kWaitDrain) &&
             wait_bar_warp(o_full(1), o1_count & 1, wc, kWaitOFull);
        if (!ok) break;
        ++x_count;
        const float2 x = xml[r_tile];
        const float m = fmaxf(m_ref, x.x), m0 = m == -INFINITY ? 0.f : m;
        a0 = ex2_approx(m_ref - m0);
        a1 = ex2_approx(x.x - m0);
        // a row without any key keeps its zeros; a NaN stays one
        l = l * a0 + x.y * a1;
        m_ref = m;
        tc_fence_after();
      }
      if (s.active(1)) ++o1_count;
      // O, 32 columns at a time; compact on purpose (this code is out of the
      // instruction caches whenever it runs).  A lane has a row, so each store
      // writes 32 lines and their number is what the loop costs: 32 bytes a lane
      // instead of 16 took short prompts (19 of up to 895 tokens, 56 heads) from 311
      // to 304 us; exchanging chunks between lanes for whole lines cost more than it
      // gave (328).
      const bool o_wide = (reinterpret_cast<uintptr_t>(args.o) & 31) == 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int token = rr / args.group;
      const long long out_row =
          (static_cast<long long>(s.r0 + token) * args.Hkv + s.head) * args.group + (rr - token * args.group);
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * ch, o);
        if (joined) {
          uint32_t o1[32];
          tmem_ld32(tmem + lane_off + C::col_o(1) + 32 * ch, o1);
          tmem_ld_wait32(o);
          reg_fence32(o1);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), a1, __uint_as_float(o[i]) * a0));
        }
        tmem_ld_wait32(o);
        if (!on || !dcheck(inside(out_row, 1, q_rows), args.status, 644)) continue;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int z = 0; z < 8; ++z)
              w[z] = pack_bf16x2(__uint_as_float(o[16 * i + 2 * z]) * inv,
                                 __uint_as_float(o[16 * i + 2 * z + 1]) * inv);
            uint16_t* dst = args.o + out_row * D + 32 * ch + 16 * i;
            if (o_wide) {
              st_global_v8(dst, w);
            } else {
              reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w[8] = {o[8 * i],     o[8 * i + 1], o[8 * i + 2], o[8 * i + 3],
                                   o[8 * i + 4], o[8 * i + 5], o[8 * i + 6], o[8 * i + 7]};
            st_global_v8(part + 8 * ch + 2 * i, w);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(o_empty(t));
      if (joined) {
        mbar_arrive(o_empty(1));
        mbar_arrive(x_empty);
      }
      if (on) {
        if (whole) args.lse[out_row] = l == 0.f ? -INFINITY : (m_ref - kLift + log2f(l)) * kLn2;
        else *part_ml = make_float2(m_ref - kLift, l);
      }
      done_seg(si);
    }
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    // ================================================================ MMA issue
    const uint32_t lead = elect_lane();
    constexpr uint32_t idesc_qk = idesc_e4m3_f32(kBM, kBN);
    constexpr uint32_t idesc_pv = idesc_f16_f32(kBM, D);
    uint32_t kc = 0, hc = 0;              // K tiles and fp16 V tiles taken so far
    uint32_t qc[2] = {0u, 0u}, pc[2] = {0u, 0u}, oc[2] = {0u, 0u};
    auto issue_s = [&](int t) {
      const uint64_t db = sdesc_codes<D>(sbase + C::kKOff + (kc % C::kKStages) * C::kCodeTile);
      const uint64_t da = sdesc_codes<D>(sbase + C::kQOff + t * C::kQBytes);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {          // the hi part's steps, then the lo part's
        const uint32_t kk = 2u * (i & (D / 32 - 1)), part = i >= D / 32 ? C::kCodeTile >> 4 : 0u;
        mma_codes(tmem + C::col_s(t), da + (kk + part), db + kk, idesc_qk, i > 0 ? 1u : 0u, lead);
      }
      commit_to(s_full(t), lead);
    };
    auto issue_pv = [&](int t, uint32_t acc) {
      const uint64_t dv = sdesc_sw128(sbase + C::kHOff + (hc & 1) * C::kHalfTile, C::kHalfChunk, 1024);
#pragma unroll
      for (int kk = 0; kk < kBN / 16; ++kk)
        mma_halves(tmem + C::col_o(t), tmem + C::col_s(t) + 8 * kk, dv + ((kk * 2048) >> 4), idesc_pv,
                   kk > 0 ? 1u : acc, lead);
    };
    auto wait_k = [&]() {
      return wait_bar_warp(k_full(kc % C::kKStages), (kc / C::kKStages) & 1, wc, kWaitKvFull);
    };
    // One segment, tiles [a, e), row tile t up to e_t.  Its bounds come
    // through a shuffle, which tells the compiler that they are the same in
    // every lane: MMAs issued under branches that it takes for divergent cost
    // their issue several times over (measured: 5500 cycles a step of 32
    // MMAs where the tensor core needs 2048).
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    auto run = [&](const int a, const int e, const int e0, const int e1) -> bool {
      if (!wait_k()) return false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if ((t ? e1 : e0) > a) {
          if (!wait_bar_warp(q_full(t), qc[t]++ & 1, wc, kWaitQFull)) return false;
          tc_fence_after();
          issue_s(t);
          if (a + 1 == (t ? e1 : e0)) commit_to(q_empty(t), lead);   // its only scores
        }
      }
      commit_to(k_empty(kc % C::kKStages), lead);
      ++kc;
      for (int j = a; j < e; ++j) {
        if (!wait_bar_warp(h_full(hc & 1), (hc >> 1) & 1, wc, kWaitDsFull)) return false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int et = t ? e1 : e0;
          // A K tile that neither row tile needs any more is taken all the same.
          if (t == 0 && j + 1 < e && !wait_k()) return false;
          if (j < et) {
            if (j == a && oc[t] > 0 && !wait_bar_warp(o_empty(t), (oc[t] - 1) & 1, wc, kWaitOFull))
              return false;
            if (!wait_bar_warp(p_full(t), pc[t]++ & 1, wc, kWaitPFull)) return false;
            tc_fence_after();
            issue_pv(t, j > a ? 1u : 0u);
            if (j + 1 == et) {
              commit_to(o_full(t), lead);
              ++oc[t];
            }
          }
          if (j + 1 < et) {
            issue_s(t);
            if (j + 2 == et) commit_to(q_empty(t), lead);
          }
        }
        commit_to(h_empty(hc & 1), lead);
        ++hc;
        if (j + 1 < e) {
          commit_to(k_empty(kc % C::kKStages), lead);
          ++kc;
        }
      }
      return true;
    };
    // A narrow part of n key tiles: tile i is slot i & 1's.
    auto run_narrow = [&](const int n) -> bool {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t < n) {
          if (!wait_k()) return false;
          if (!wait_bar_warp(q_full(t), qc[t]++ & 1, wc, kWaitQFull)) return false;
          tc_fence_after();
          issue_s(t);
          if (t + 2 >= n) commit_to(q_empty(t), lead);
          commit_to(k_empty(kc % C::kKStages), lead);
          ++kc;
        }
      }
      for (int i = 0; i < n; i += 2) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (i + t < n) {
            if (!wait_bar_warp(h_full(hc & 1), (hc >> 1) & 1, wc, kWaitDsFull)) return false;
            if (i == 0 && oc[t] > 0 && !wait_bar_warp(o_empty(t), (oc[t] - 1) & 1, wc, kWaitOFull))
              return false;
            if (i + t + 2 < n && !wait_k()) return false;
            if (!wait_bar_warp(p_full(t), pc[t]++ & 1, wc, kWaitPFull)) return false;
            tc_fence_after();
            issue_pv(t, i > 0 ? 1u : 0u);
            commit_to(h_empty(hc & 1), lead);
            ++hc;
            if (i + t + 2 < n) {
              issue_s(t);
              if (i + t + 4 >= n) commit_to(q_empty(t), lead);
              commit_to(k_empty(kc % C::kKStages), lead);
              ++kc;
            } else {
              commit_to(o_full(t), lead);
              ++oc[t];
            }
          }
        }
      }
      return true;
    };
    for (uint32_t si = 0; wait_seg(si); ++si) {
      const Seg& s = seg_at(si);
      const int flags = uniform(s.flags), a = uniform(s.a), e = uniform(s.e), e0 = uniform(s.e0);
      if (flags & Seg::kLast) break;
      done_seg(si);
      if (flags & Seg::kNarrow) {
        if (!run_narrow(e - a)) break;
      } else {
        if (!run(a, e, e0, e)) break;
      }
    }
    // No MMA may still be running when TMEM is released.
    commit_to(mma_done, lead);
    mbar_wait_drain(mma_done, 0);
    __syncwarp();
  } else if (warp == kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    // ================================================================ TMA producer
    const int per_log = 7 - args.page_shift, per = 1 << per_log;   // pages per key tile
    const uint32_t page_bytes = static_cast<uint32_t>(D) << args.page_shift;
    uint32_t kn = 0, vn = 0;              // K and V tiles asked for so far
    uint32_t qn[2] = {0u, 0u};            // and Q tiles
    bool ok = true;
    wait_for_parent();                    // q_codes
    for (uint32_t si = 0; ok && wait_seg(si); ++si) {
      const Seg s = seg_at(si);
      if (s.flags & Seg::kLast) break;
      done_seg(si);
      int base = s.a << per_log;          // 32 pages here, the next 32 on the way
      int cur = page_of_lane(args, s.b, s.len, base), nxt = page_of_lane(args, s.b, s.len, base + 32);
      for (int j = s.a; j < s.e; ++j) {
        if ((j << per_log) >= base + 32) {
          base += 32;
          cur = nxt;
          nxt = page_of_lane(args, s.b, s.len, base + 32);
        }
        int pid[4];
        uint32_t mask = 0u, bytes = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pid[i] = -1;
          if (i < per) {
            const int p = (j << per_log) + i;
            pid[i] = __shfl_sync(0xffffffffu, cur, p - base);
            if (pid[i] < 0 || pid[i] >= args.pages) {
              if (lane == 0 && (static_cast<long long>(p) << args.page_shift) < s.len)
                record_bad_index(args.status, kSitePage);
              pid[i] = -1;
            } else {
              mask |= ((1u << (4 >> per_log)) - 1u) << (i * (4 >> per_log));
              bytes += page_bytes;
            }
          }
        }
        const uint32_t ks = kn % C::kKStages, vs = vn % C::kVStages;
        if (kn >= C::kKStages &&
            !wait_bar_warp(k_empty(ks), (kn / C::kKStages - 1) & 1, wc, kWaitKvEmpty)) {
          ok = false;
          break;
        }
        ok = dcheck(in_range(sbase + C::kKOff + ks * C::kCodeTile, C::kCodeTile, sbase + C::kKOff, sbase + C::kVOff) &&
                        in_range(sbase + C::kVOff + vs * C::kCodeTile, C::kCodeTile, sbase + C::kVOff, sbase + C::kHOff) &&
                        bytes <= static_cast<uint32_t>(C::kCodeTile) && inside(s.head, 1, args.Hkv),
                    args.status, 645);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(k_full(ks), bytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (pid[i] >= 0)
              tma_load_3d(sbase + C::kKOff + ks * C::kCodeTile + i * page_bytes, &tm_k, k_full(ks), 0,
                          s.head << args.page_shift, pid[i]);
        }
        ++kn;
        if (j == s.a) {
          // Q's two parts, up to 128 rows each; rows past the unit's last
          // keep what the buffer held (their results go nowhere).
#pragma unroll 1
          for (int t = 0; t < 2 && ok; ++t) {
            if (!s.active(t)) continue;
            if (qn[t] > 0) ok = wait_bar_warp(q_empty(t), (qn[t] - 1) & 1, wc, kWaitQFull);
            if (!ok) break;
            const int first = s.row(t, 0);
            const uint32_t nb = static_cast<uint32_t>(min(kBM, s.n * args.group - first)) * D;
            const uint8_t* src = args.q_codes + (s.q_row(args) + first) * D;
            const uint32_t dst = sbase + C::kQOff + t * C::kQBytes;
            ok = dcheck(first < s.n * args.group && nb <= static_cast<uint32_t>(C::kCodeTile) &&
                            in_range(dst, C::kCodeTile + nb, sbase + C::kQOff, sbase + C::kKOff) &&
                            inside((s.q_row(args) + first) * D, nb, q_rows * D),
                        args.status, 646);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(q_full(t), 2 * nb);
              bulk_load_1d(dst, src, nb, q_full(t));
              bulk_load_1d(dst + C::kCodeTile, src + args.q_lo, nb, q_full(t));
            }
            ++qn[t];
          }
          if (!ok) break;
        }
        if (vn >= C::kVStages &&
            !wait_bar_warp(v_empty(vs), (vn / C::kVStages - 1) & 1, wc, kWaitKvEmpty)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          valid[vs] = mask;
          mbar_arrive_expect_tx(v_full(vs), bytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (pid[i] >= 0)
              tma_load_3d(sbase + C::kVOff + vs * C::kCodeTile + i * page_bytes, &tm_v, v_full(vs), 0,
                          s.head << args.page_shift, pid[i]);
        }
        ++vn;
      }
    }
    // Every copy this warp started must have landed before the CTA exits.
    for (uint32_t r = kn > C::kKStages ? kn - C::kKStages : 0; r < kn; ++r)
      mbar_wait_drain(k_full(r % C::kKStages), (r / C::kKStages) & 1);
    for (uint32_t r = vn > C::kVStages ? vn - C::kVStages : 0; r < vn; ++r)
      mbar_wait_drain(v_full(r % C::kVStages), (r / C::kVStages) & 1);
    for (int t = 0; t < 2; ++t)
      if (qn[t] > 0) mbar_wait_drain(q_full(t), (qn[t] - 1) & 1);
    __syncwarp();
  } else if (warp < kConvWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    // ================================================================ schedule
    if (warp == kWalkWarp) {
      const long long j0 = cta_first(W, G, cta), j1 = cta_first(W, G, cta + 1);
      Walker walk(args, pre, j0, j1);
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
        if (i >= kSegs && !wait_bar_warp(seg_empty(i), (i / kSegs - 1) & 1, wc, kWaitSegment)) {
          any = false;
          break;
        }
        if (lane == 0) {
          const_cast<Seg&>(seg_at(i)) = x;
          mbar_arrive(seg_full(i));
        }
        __syncwarp();
        if (!more) break;
        // The segment's first scales, which the softmax warps will ask for, to L1.
        const int pid = page_of_lane(args, x.b, x.len, x.a << (7 - args.page_shift));
        if (pid >= 0 && pid < args.pages) {
          const long long sc = static_cast<long long>(pid) * args.Hkv + x.head;
          prefetch_l1(args.k_scale + sc);
          prefetch_l1(args.v_scale + sc);
        }
      }
      if (lane == 0) {
        // What is to be joined: the unit that this CTA starts and others go
        // on with (its last one).
        const bool shared_unit = any && (s.flags & (Seg::kStarts | Seg::kEnds)) == Seg::kStarts;
        args.rec[2 * cta] = shared_unit ? make_int4(s.r0, s.n, s.rb, s.head) : make_int4(0, 0, 0, 0);
        if (shared_unit)
          args.rec[2 * cta + 1] = make_int4(cta_of(W, G, j1 - (s.e - s.a) + s.nt - 1),
                                            static_cast<int>(W), static_cast<int>(W >> 32), 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ================================================================ V to fp16
    // The fp16 tile is laid out as the P V product reads it: two chunks of 64
    // columns, rows of 128 bytes with the 128-byte swizzle.  A thread takes
    // one 16-byte chunk of codes (16 columns) of a row at a time, eight
    // neighbouring lanes two rows of four, so that their stores meet
    // different banks.
    constexpr int CH = D / 16;            // 16-byte chunks of a code row
    constexpr int kIter = kBN * CH / 128;
    const int ct = tid - 32 * kConvWarp0;   // 0 .. 127
    auto row_of = [](int id) { return D == 128 ? (id >> 4) * 2 + (id >> 2 & 1) : id >> 2; };
    auto chunk_of = [](int id) { return D == 128 ? (id & 3) | (id >> 3 & 1) << 2 : id & 3; };
    uint32_t cnt = 0;
    bool ok = true;
    for (uint32_t si = 0; ok && wait_seg(si); ++si) {
      const int a = seg_at(si).a, e = seg_at(si).e, len = seg_at(si).len, flags = seg_at(si).flags;
      if (flags & Seg::kLast) break;
      done_seg(si);
      for (int j = a; j < e; ++j) {
        const uint32_t st = cnt % C::kVStages, hs = cnt & 1;
        if (!wait_bar_warp(v_full(st), (cnt / C::kVStages) & 1, wc, kWaitKvFull) ||
            (cnt > 1 && !wait_bar_warp(h_empty(hs), ((cnt >> 1) - 1) & 1, wc, kWaitMmaDone))) {
          ok = false;
          break;
        }
        const uint32_t src = sbase + C::kVOff + st * C::kCodeTile;
        const uint32_t dst = sbase + C::kHOff + hs * C::kHalfTile;
        const uint32_t mask = valid[st];
        const int left = len - j * kBN;            // keys of the tile that exist
        const bool edge = left < kBN || mask != 0xfu;
        // Not unrolled: the kernel's roles share the instruction caches, and
        // 6 KB of straight-line conversion here made every one of them wait
        // for instructions (measured: 2 x 2048 rows on 16384 keys 1142 us
        // unrolled, 767 us so).
#pragma unroll 1
        for (int i0 = 0; i0 < kIter; i0 += 2) {
          uint4 w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int id = ct + 128 * (i0 + i), row = row_of(id), c = chunk_of(id);
            w[i] = ld_shared_v4(src + code_off<D>(row, c));
            // Slots behind the end and pages that were not loaded hold
            // anything, NaN codes too.
            if (edge && (row >= left || !(mask >> (row >> 5) & 1u))) w[i] = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int id = ct + 128 * (i0 + i), row = row_of(id), c = chunk_of(id);
            const uint32_t base = dst + (c >> 2) * C::kHalfChunk + row * 128;
            const int c2 = 2 * (c & 3);            // 16-byte chunk of the fp16 row
            if (!dcheck(in_range(src + code_off<D>(row, c), 16, sbase + C::kVOff, sbase + C::kHOff) &&
                            in_range(base, 128, sbase + C::kHOff, sbase + C::kBarOff),
                        args.status, 647))
              continue;
            uint4 x, y;
            e4m3x4_to_f16x4(w[i].x, x.x, x.y);
            e4m3x4_to_f16x4(w[i].y, x.z, x.w);
            e4m3x4_to_f16x4(w[i].z, y.x, y.y);
            e4m3x4_to_f16x4(w[i].w, y.z, y.w);
            st_shared_v4(base + ((c2 ^ (row & 7)) << 4), x.x, x.y, x.z, x.w);
            st_shared_v4(base + (((c2 + 1) ^ (row & 7)) << 4), y.x, y.y, y.z, y.w);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(h_full(hs));
          mbar_arrive(v_empty(st));
        }
        ++cnt;
      }
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

// Splits the call's queries: row x = q * 2^-e, its largest entry in [224, 448]
// (up to 448 where the mantissa allows), into hi = e4m3(x) and lo =
// e4m3(x - hi).  Rows go to where the products read them: those of a sequence and
// kv head in one run, (token, query head) order, 16-byte chunks swizzled as in
// shared memory, so that a tile is one plain copy.  Bound: 2 d bytes in and out
// a row.  A thread takes 16 columns of kSplitRows rows of one token, so that the
// search for its sequence is shared and the loads go out together: 19 prompts with
// 160 MB of queries took 298 us with one row a thread (55 of them here), 288 with
// two, 285 with four, 290 with eight.
constexpr int kSplitRows = 4;

template <int D>
__global__ void __launch_bounds__(256) split_kernel(const __grid_constant__ CacheAttnArgs a) {
  allow_child();
  constexpr int kLanes = D / 16;          // 16 columns each
  const int Hq = a.Hkv * a.group, groups = (Hq + kSplitRows - 1) / kSplitRows;
  const int item = static_cast<int>((static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / kLanes);
  const int c = threadIdx.x % kLanes;
  const int token = item / groups, h0 = (item - token * groups) * kSplitRows;
  if (token >= a.s.T) return;              // whole groups of lanes
  // the token's sequence: a guess for sequences of equal rows, else a search
  int b = static_cast<int>(static_cast<long long>(token) * a.s.B / a.s.T);
  if (token < __ldg(a.s.q_start + b) || token >= __ldg(a.s.q_start + b + 1)) {
    b = 0;
    for (int hi = a.s.B; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (__ldg(a.s.q_start + mid) <= token) b = mid; else hi = mid;
    }
  }
  const SeqInfo q = seq_info(a.s, b, a.page_shift);
  if (token < q.r0 || token >= q.r0 + q.n) return;   // behind the last sequence
  uint4 w[kSplitRows][2];
#pragma unroll
  for (int k = 0; k < kSplitRows; ++k) {
    const uint4* p = reinterpret_cast<const uint4*>(a.q + token * a.q_row + min(h0 + k, Hq - 1) * D + 16 * c);
    w[k][0] = __ldg(p);
    w[k][1] = __ldg(p + 1);
  }
  // a row's lanes are neighbours, and all of them are here
  const unsigned int lanes = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
  for (int k = 0; k < kSplitRows; ++k) {
    if (h0 + k >= Hq) break;
    const uint32_t u[8] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w,
                           w[k][1].x, w[k][1].y, w[k][1].z, w[k][1].w};
    uint32_t mx = 0u;                        // the largest magnitude's bits
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) mx = max(mx, __shfl_xor_sync(lanes, mx, off));
    const float factor = query_factor(mx);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int z = 0; z < 4; ++z) split_query4(u[2 * z], u[2 * z + 1], factor, hi[z], lo[z]);
    const int hq = h0 + k, head = hq / a.group;
    const int rr = (token - q.r0) * a.group + (hq - head * a.group);
    const long long out = (static_cast<long long>(q.r0) * a.Hkv + static_cast<long long>(head) * q.n) * a.group + rr;
    // swizzle of the row's place in its tile (tiles start at multiples of 128 rows)
    if (!dcheck(inside(out, 1, static_cast<long long>(a.s.T) * Hq) &&
                    inside(out * D - static_cast<long long>(rr & 7) * D + code_off<D>(rr & 7, c), 16,
                           static_cast<long long>(a.s.T) * Hq * D),
                a.status, 648))
      continue;
    uint8_t* dst = a.q_codes + out * D - static_cast<long long>(rr & 7) * D + code_off<D>(rr & 7, c);
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(dst + a.q_lo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (c == 0) a.q_scale[out] = query_scale(mx);
  }
}

template <int D>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                     cudaStream_t stream) {
  auto kern = chunk_kernel<D>;
  const int smem = ChunkCfg<D>::kSmemFixed + (a.s.B + 1) * 4;
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  // The register split inside the kernel is only valid for this launch size.
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const long long lanes =
      static_cast<long long>(a.s.T) * ((a.Hkv * a.group + kSplitRows - 1) / kSplitRows) * (D / 16);
  split_kernel<D><<<static_cast<unsigned>((lanes + 255) / 256), 256, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_child(kern, a.grid, kThreads, smem, stream, tk, tv, a)) != cudaSuccess) return e;
  return launch_cache_join(D, kUnitRows, a, stream);
}

}  // namespace

cudaError_t launch_cache_chunk(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CacheAttnArgs& a, cudaStream_t stream) {
  return d == 64 ? launch_t<64>(tk, tv, a, stream) : launch_t<128>(tk, tv, a, stream);
}

}  // namespace fattn
