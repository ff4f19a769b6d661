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
//     product would, and K needs no conversion.
//   O += P V    in fp16 (kind::f16): probabilities to fp16 in tensor memory
//     (one rounding, 2^-11), V's codes to fp16, exactly, by two converter
//     warps between the TMA ring and the MMA's tiles.  An e4m3 P would lose
//     2^-4 of every probability; splitting P as Q is would cost the softmax
//     warps three conversions per pair, and they set the pace already.
//
// Softmax with the page scales inside, as in the kernel for few rows: with
// c_p = scale log2(e) 2^e(row) kscale_p and l_p = log2 vscale_p,
//   x_j = c_p s_j + l_p,  P'_j = 2^(x_j - m),  l = sum_p 2^(-l_p) sum P'.
// A page is at least 32 tokens, so c and l_p are constant over each 32-column
// TMEM load and the row maximum comes from the load itself (tcgen05.ld.red).
// The reference m moves only when a row's maximum passes it by more than 8
// (fp16 holds 2^8 times a probability easily).
//
// Work split: the key tiles of all units, in order, are dealt to the CTAs in
// equal contiguous shares, whatever the sequences' lengths and however many
// tiles causality cuts off; units that CTAs share are joined from partial
// results in a second kernel, in order.
//
// Warps: 0-3 softmax of row tile 0, 4-7 of row tile 1 (they also bring their
// rows of Q in, as hi and lo parts), 8 tensor memory and MMA issue, 9 TMA, 10-11
// conversion of V.  TMEM: S_t [128 t, 128 t + 128), P aliases S, O_t at 256 + d t.
#include <cuda_fp16.h>

#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kBM = 128;              // rows per tile
constexpr int kBN = 128;              // keys per tile
constexpr int kUnitRows = kChunkRows;
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kTau = 8.f;
// The same split as the dense forward: 128 x 72 + 256 x 216 = 384 x 168.
constexpr int kLaunchRegs = 168;
constexpr int kCtrlRegs = 72;
constexpr int kSoftmaxRegs = 216;
static_assert(128 * kCtrlRegs + 256 * kSoftmaxRegs == kThreads * kLaunchRegs, "register split");
static_assert(kUnitRows == 2 * kBM, "rows of a unit");

template <int D>
struct ChunkCfg {
  static constexpr int kCodeTile = kBN * D;              // e4m3 tile: rows of D bytes, swizzled by D
  static constexpr int kQBytes = 2 * kCodeTile;          // hi, lo of one row tile
  static constexpr int kHalfTile = kBN * D * 2;          // fp16 V tile
  static constexpr int kHalfChunk = kBN * 128;           // 64 columns of it
  static constexpr int kKStages = 3;
  static constexpr int kVStages = 2;                     // codes; two fp16 tiles follow
  static constexpr int kQOff = 0;
  static constexpr int kKOff = 2 * kQBytes;
  static constexpr int kVOff = kKOff + kKStages * kCodeTile;
  static constexpr int kHOff = kVOff + kVStages * kCodeTile;
  static constexpr int kBarOff = kHOff + 2 * kHalfTile;
  // k_full[] k_empty[] v_full[] v_empty[] h_full[2] h_empty[2] q_full[2]
  // s_full[2] p_full[2] o_full[2] o_empty[2] mma_done
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 15;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;   // tmem, abort, valid[kVStages]
  static constexpr int kPreOff = kMiscOff + 64;             // [B + 1] int
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

// kind::f16 with fp16 A and B (format code 0), fp32 D; B is MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Key tiles that the rows [256 rb, 256 rb + rows) of a sequence need.  Row R
// sees pos0 + R / g + 1 keys, so rows before row E see at most pos0 + ceil(E / g).
// At least one, so that rows that see nothing are written, too.
__device__ __forceinline__ int tiles_of(const CacheAttnArgs& a, int n, int len, int rb, int rows) {
  const long long g = a.group;
  const long long all = (len + kBN - 1) / kBN;
  if (!a.causal) return static_cast<int>(max(1ll, all));
  const long long end = min(n * g, static_cast<long long>(rb) * kUnitRows + rows);
  const long long keys = (len - n) * g + end;
  const long long nt = keys <= 0 ? 0 : (keys + kBN * g - 1) / (kBN * g);
  return static_cast<int>(max(1ll, min(all, nt)));
}

// One CTA's part of a unit: key tiles [a, e) for the rows from 256 rb of a
// sequence; row tile t has tiles up to e_t[t] (a where it has none).
struct Seg {
  int b, rb, head;
  int r0, n, len;
  int a, e, nt;
  int e_t[2];
  bool starts, ends;
};

// Walks a CTA's share; every warp that needs it runs its own, converged.
struct Walker {
  const CacheAttnArgs& a;
  const int* pre;           // key tiles before each sequence
  long long left;           // tiles still to walk
  int b, rb, head, at, nt, nrb;
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
          i < nrb ? static_cast<long long>(tiles_of(a, q.n, q.len, i, kUnitRows)) * a.Hkv : 0;
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
    head = static_cast<int>(rem / nt);
    at = static_cast<int>(rem - static_cast<long long>(head) * nt);
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (left <= 0) return false;
    if (at == nt) {
      at = 0;
      if (++head == a.Hkv) {
        head = 0;
        if (++rb == nrb) {
          rb = 0;
          // tiles are left, so a sequence with rows follows
          do {
            if (++b >= a.s.B) return false;
            load_seq();
          } while (q.n == 0);
        }
        nt = tiles_of(a, q.n, q.len, rb, kUnitRows);
      }
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
    s.starts = at == 0;
    s.ends = s.e == nt;
    const bool second = static_cast<long long>(rb) * kUnitRows + kBM <
                        static_cast<long long>(q.n) * a.group;
    s.e_t[0] = max(s.a, min(s.e, tiles_of(a, q.n, q.len, rb, kBM)));
    s.e_t[1] = second ? s.e : s.a;
    left -= s.e - s.a;
    at = s.e;
    return true;
  }
};

// 32 pages of a sequence, one per lane.
struct Window {
  int base, pid;
  __device__ __forceinline__ void load(const CacheAttnArgs& a, const Seg& s, int first) {
    base = first;
    pid = -1;
    const int p = first + static_cast<int>(threadIdx.x & 31);
    if ((static_cast<long long>(p) << a.page_shift) < s.len) {
      pid = __ldg(a.s.table + static_cast<long long>(s.b) * a.s.max_pages + p);
      if (pid < 0 || pid >= a.pages) {
        record_bad_index(a.status, kSitePage);
        pid = -1;
      }
    }
  }
};

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
  const uint32_t mma_done = rest + 112u;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile uint32_t* valid = misc + 2;   // per V stage: which 32-key groups were loaded
  int* pre = reinterpret_cast<int*>(smem + C::kPreOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, G = args.grid;

  if (tid == 0) {
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(h_full(t), 2);
      mbar_init(h_empty(t), 1);
      mbar_init(q_full(t), 4);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 128);
      mbar_init(o_full(t), 1);
      mbar_init(o_empty(t), 128);
    }
    mbar_init(mma_done, 1);
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
  // ---- key tiles before each sequence
  {
    __shared__ long long wtot[kThreads / 32];
    const int per = (args.s.B + kThreads - 1) / kThreads;
    const int b0 = min(args.s.B, tid * per), b1 = min(args.s.B, b0 + per);
    auto weight = [&](int b) -> long long {
      const SeqInfo q = seq_info(args.s, b, args.page_shift);
      if (!q.ok && cta == 0) record_bad_index(args.status, kSiteSeqStart);
      const int nrb = static_cast<int>((static_cast<long long>(q.n) * args.group + kUnitRows - 1) / kUnitRows);
      long long w = 0;
      for (int i = 0; i < nrb; ++i) w += tiles_of(args, q.n, q.len, i, kUnitRows);
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
    if (tid == kThreads - 1) pre[args.s.B] = static_cast<int>(at + sum);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const WaitCtx wc{args.wait_budget, reinterpret_cast<volatile uint32_t*>(&misc[1]), args.status};
  const long long W = pre[args.s.B];
  const long long j0 = cta_first(W, G, cta), j1 = cta_first(W, G, cta + 1);

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ================================================================ softmax
    const int t = warp >> 2;              // row tile
    const int wq = warp & 3;
    const int r_tile = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    const uint32_t q_smem = sbase + C::kQOff + t * C::kQBytes;
    const int pages_log = 7 - args.page_shift;   // log2 of the pages per key tile
    uint32_t s_count = 0, o_count = 0;
    bool ok = true;

    // This thread's row of the segment's Q, split into e4m3 parts; returns
    // log2(e) * scale times the power of two that was taken out.
    auto load_q = [&](const Seg& s) -> float {
      const long long rr = static_cast<long long>(s.rb) * kUnitRows + t * kBM + r_tile;
      const bool on = rr < static_cast<long long>(s.n) * args.group;
      uint4 w[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (on) {
        const int token = static_cast<int>(rr / args.group);
        const uint4* p = reinterpret_cast<const uint4*>(
            args.q + (s.r0 + token) * args.q_row +
            (static_cast<long long>(s.head) * args.group + (rr - static_cast<long long>(token) * args.group)) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = __ldg(p + i);
      }
      uint32_t mx = 0u;                  // largest magnitude's bf16 bits
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int z = 0; z < 4; ++z) mx = max(mx, max(u[z] & 0x7fffu, (u[z] >> 16) & 0x7fffu));
      }
      // x = q * 2^(8 - E) <= 448 where the mantissa is at most 1.75, one less above
      const int e = static_cast<int>(mx >> 7) - 127 - 8 + ((mx & 0x7fu) > 0x60u ? 1 : 0);
      const int ec = max(-126, min(126, e));
      // a row with an infinity or a NaN becomes NaN
      const float down = mx >= 0x7f80u ? __int_as_float(0x7fffffff) : exp2i(-ec);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {   // 16 columns: one 16-byte chunk of codes
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint4 v = w[2 * i + (z >> 1)];
          const uint32_t a0 = z & 1 ? v.z : v.x, a1 = z & 1 ? v.w : v.y;
          const float x0 = __uint_as_float(a0 << 16) * down, x1 = __uint_as_float(a0 & 0xffff0000u) * down;
          const float x2 = __uint_as_float(a1 << 16) * down, x3 = __uint_as_float(a1 & 0xffff0000u) * down;
          hi[z] = pack_e4m3x4(x0, x1, x2, x3);
          const float2 h0 = e4m3x2_to_f32x2(hi[z]), h1 = e4m3x2_to_f32x2(hi[z] >> 16);
          lo[z] = pack_e4m3x4(x0 - h0.x, x1 - h0.y, x2 - h1.x, x3 - h1.y);
        }
        st_shared_v4(q_smem + code_off<D>(r_tile, i), hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(q_smem + C::kCodeTile + code_off<D>(r_tile, i), lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(t));
      return args.scale_log2 * exp2i(ec);
    };

    Walker walk(args, pre, j0, j1);
    Seg s{}, sn{};
    bool more = walk.next(sn);
    float c_row = 0.f;
    if (more && sn.e_t[t] > sn.a) c_row = load_q(sn);
    while (ok && more) {
      s = sn;
      more = walk.next(sn);
      const bool whole = s.starts && s.ends;
      const long long rr = static_cast<long long>(s.rb) * kUnitRows + t * kBM + r_tile;
      const bool on = rr < static_cast<long long>(s.n) * args.group;
      const int token = on ? static_cast<int>(rr / args.group) : 0;
      // Keys the row sees.  Rows past the unit's last see all (their queries
      // are zero), so that they need no mask.
      const int lim = !on || !args.causal ? s.len : max(0, min(s.len, s.len - s.n + token + 1));
      float m_ref = -INFINITY, l = 0.f;
      const float c0 = c_row;
      const int nj = s.e_t[t];
      Window win;
      float w_ks = 0.f, w_lv = 0.f;
      auto load_window = [&](int first) {
        win.load(args, s, first);
        w_ks = 0.f;
        w_lv = 0.f;
        if (win.pid >= 0) {
          const long long sc = static_cast<long long>(win.pid) * args.Hkv + s.head;
          w_ks = __ldg(args.k_scale + sc);
          w_lv = static_cast<float>(scale_exp(__ldg(args.v_scale + sc)));
        }
      };
      if (s.a < nj) load_window(s.a << pages_log);
      for (int j = s.a; j < nj; ++j) {
        if (((j + 1) << pages_log) - win.base > 32) load_window(j << pages_log);
        float cg[4], lg[4];               // per 32 columns: exponent factor, log2 of the V scale
        bool hole = false;                // a page that is not there
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int p = ((j * kBN + 32 * g) >> args.page_shift) - win.base;
          const float ks = __shfl_sync(0xffffffffu, w_ks, p);
          lg[g] = __shfl_sync(0xffffffffu, w_lv, p);
          // positive, so that a masked score stays -inf (|S| < 2^26: what is
          // lost is far below the last bit of a probability)
          cg[g] = fmaxf(c0 * ks, 1e-37f);
          hole |= __shfl_sync(0xffffffffu, win.pid, p) < 0;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(t), s_count & 1, wc, kWaitSFull));
        if (!ok) break;
        ++s_count;
        tc_fence_after();
        uint32_t s0[32], s1[32], s2[32], s3[32];
        float mg[4];
        tmem_ld32_max(tS + 0, s0, mg[0]);
        tmem_ld32_max(tS + 32, s1, mg[1]);
        tmem_ld32_max(tS + 64, s2, mg[2]);
        tmem_ld32_max(tS + 96, s3, mg[3]);
        tmem_ld_wait32(s0);
        reg_fence32(s1);
        reg_fence32(s2);
        reg_fence32(s3);
#pragma unroll
        for (int g = 0; g < 4; ++g) reg_fence1(mg[g]);
        uint32_t* sv[4] = {s0, s1, s2, s3};
        const int kv0 = j * kBN;
        if (__any_sync(0xffffffffu, kv0 + kBN > lim || hole)) {
          const int lt = lim - kv0;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int p = ((kv0 + 32 * g) >> args.page_shift) - win.base;
            const int lh = __shfl_sync(0xffffffffu, win.pid, p) < 0 ? 0 : lt;
            mg[g] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (g * 32 + i >= lh) sv[g][i] = __float_as_uint(-INFINITY);
              mg[g] = fmaxf(mg[g], __uint_as_float(sv[g][i]));
            }
          }
        }
        float x[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) x[g] = fmaf(mg[g], cg[g], lg[g]);
        const float m_new = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        const bool need = m_new > m_ref + kTau;
        const bool rescale = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (rescale) {
          alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
          if (need) m_ref = m_new;
          l *= alpha;
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        float rs[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t pk[16];
          uint64_t e2 = 0ull;
          const uint64_t c2 = splat2(cg[g]);
          const uint64_t nm2 = splat2(lg[g] - m_use);
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
          rs[g] = (__uint_as_float(u0) + __uint_as_float(u1)) * ex2_approx(-lg[g]);
        }
        if (rescale && j > s.a) {
          // P V of the last tile has completed: it was issued before this S.
          uint32_t o[D / 32][32];
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) tmem_ld32(tO + 32 * ch, o[ch]);
          tmem_ld_wait32(o[0]);
#pragma unroll
          for (int ch = 1; ch < D / 32; ++ch) reg_fence32(o[ch]);
          const uint64_t a2 = splat2(alpha);
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              unpack2(fmul2(pack2(o[ch][2 * i], o[ch][2 * i + 1]), a2), o[ch][2 * i],
                      o[ch][2 * i + 1]);
            tmem_st32(tO + 32 * ch, o[ch]);
          }
        }
        l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(t));
      }
      if (!ok) break;
      // The next segment's Q: this tile's last S has been read, so its
      // product has left the buffer.
      if (more && sn.e_t[t] > sn.a) c_row = load_q(sn);

      // ---- results
      const long long slot = 2ll * cta + (s.starts ? 1 : 0);
      if (nj == s.a) {
        // Nothing for this row tile here (causality, or no rows at all): an
        // empty part, where the unit has other parts.
        if (!whole && on) {
          float4* p = reinterpret_cast<float4*>(args.part_o + (slot * kUnitRows + t * kBM + r_tile) * D);
          for (int i = 0; i < D / 4; ++i) p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          args.part_ml[slot * kUnitRows + t * kBM + r_tile] = make_float2(-INFINITY, 0.f);
        }
        continue;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(o_full(t), o_count & 1, wc, kWaitOFull));
      if (!ok) break;
      ++o_count;
      tc_fence_after();
      if (!whole) {
        float4* p = reinterpret_cast<float4*>(args.part_o + (slot * kUnitRows + t * kBM + r_tile) * D);
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * ch, o);
          tmem_ld_wait32(o);
          if (on) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              p[8 * ch + i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                          __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          }
        }
        tc_fence_before();
        mbar_arrive(o_empty(t));
        if (on) args.part_ml[slot * kUnitRows + t * kBM + r_tile] = make_float2(m_ref, l);
        continue;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t pw[D / 2];
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * ch, o);
        tmem_ld_wait32(o);
        const uint64_t i2 = splat2(inv);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t y0, y1;
          unpack2(fmul2(pack2(o[2 * i], o[2 * i + 1]), i2), y0, y1);
          pw[16 * ch + i] = pack_bf16x2(__uint_as_float(y0), __uint_as_float(y1));
        }
      }
      tc_fence_before();
      mbar_arrive(o_empty(t));
      // Whole 128-byte lines: 8 lanes exchange 16-byte chunks, an 8 x 8
      // transpose per 128 bytes, so that a warp store writes 4 lines.
      const int li = lane & 7;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
#pragma unroll
        for (int dd = 4; dd >= 1; dd >>= 1) {
          const bool up = (li & dd) != 0;
#pragma unroll
          for (int jj = 0; jj < 8; ++jj) {
            if (jj & dd) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t lo = pw[4 * (8 * h + jj) + q];
              const uint32_t hi = pw[4 * (8 * h + jj + dd) + q];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, dd);
              pw[4 * (8 * h + jj) + q] = up ? got : lo;
              pw[4 * (8 * h + jj + dd) + q] = up ? hi : got;
            }
          }
        }
      }
      const long long out_row =
          on ? (static_cast<long long>(s.r0 + token) * args.Hkv + s.head) * args.group +
                   (rr - static_cast<long long>(token) * args.group)
             : -1;
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        const long long row = __shfl_sync(0xffffffffu, out_row, (lane & ~7) + jj);
        if (row < 0) continue;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          __stcs(reinterpret_cast<uint4*>(args.o + row * D + 64 * h + 8 * li),
                 make_uint4(pw[4 * (8 * h + jj)], pw[4 * (8 * h + jj) + 1], pw[4 * (8 * h + jj) + 2],
                            pw[4 * (8 * h + jj) + 3]));
      }
      if (on) args.lse[out_row] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
    }
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    // ================================================================ MMA issue
    constexpr uint32_t idesc_qk = idesc_e4m3_f32(kBM, kBN);
    constexpr uint32_t idesc_pv = idesc_f16_f32(kBM, D);
    uint32_t kc = 0, hc = 0;              // K tiles and fp16 V tiles taken so far
    uint32_t qc[2] = {0u, 0u}, pc[2] = {0u, 0u}, oc[2] = {0u, 0u};
    auto issue_s = [&](int t) {
      const uint64_t db = sdesc_codes<D>(sbase + C::kKOff + (kc % C::kKStages) * C::kCodeTile);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint64_t da = sdesc_codes<D>(sbase + C::kQOff + t * C::kQBytes + part * C::kCodeTile);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_ss_f8_w(tmem + C::col_s(t), da + 2 * kk, db + 2 * kk, idesc_qk, part + kk > 0 ? 1u : 0u);
      }
      mma_commit_w(s_full(t));
    };
    auto issue_pv = [&](int t, uint32_t acc) {
      const uint64_t dv = sdesc_sw128(sbase + C::kHOff + (hc & 1) * C::kHalfTile, C::kHalfChunk, 1024);
#pragma unroll
      for (int kk = 0; kk < kBN / 16; ++kk)
        mma_ts_w(tmem + C::col_o(t), tmem + C::col_s(t) + 8 * kk, dv + ((kk * 2048) >> 4), idesc_pv,
                 kk > 0 ? 1u : acc);
    };
    auto wait_k = [&]() {
      return mbar_wait_warp(k_full(kc % C::kKStages), (kc / C::kKStages) & 1, wc, kWaitKvFull);
    };
    Walker walk(args, pre, j0, j1);
    Seg s;
    bool ok = true;
    while (ok && walk.next(s)) {
      // first scores of both tiles
      if (!(ok = wait_k())) break;
      for (int t = 0; t < 2 && ok; ++t) {
        if (s.e_t[t] <= s.a) continue;
        ok = mbar_wait_warp(q_full(t), qc[t]++ & 1, wc, kWaitQFull);
        if (!ok) break;
        tc_fence_after();
        issue_s(t);
      }
      if (!ok) break;
      mma_commit_w(k_empty(kc % C::kKStages));
      ++kc;
      for (int j = s.a; j < s.e && ok; ++j) {
        bool k_ready = false;
        ok = mbar_wait_warp(h_full(hc & 1), (hc >> 1) & 1, wc, kWaitDsFull);
        for (int t = 0; t < 2 && ok; ++t) {
          if (j < s.e_t[t]) {
            if (j == s.a && oc[t] > 0) {
              ok = mbar_wait_warp(o_empty(t), (oc[t] - 1) & 1, wc, kWaitOFull);
              if (!ok) break;
            }
            ok = mbar_wait_warp(p_full(t), pc[t]++ & 1, wc, kWaitPFull);
            if (!ok) break;
            tc_fence_after();
            issue_pv(t, j > s.a ? 1u : 0u);
            if (j + 1 == s.e_t[t]) {
              mma_commit_w(o_full(t));
              ++oc[t];
            }
          }
          if (j + 1 < s.e_t[t]) {
            if (!k_ready) {
              if (!(ok = wait_k())) break;
              k_ready = true;
              tc_fence_after();
            }
            issue_s(t);
          }
        }
        if (!ok) break;
        mma_commit_w(h_empty(hc & 1));
        ++hc;
        if (j + 1 < s.e) {
          // Both tiles may be done with their keys before the unit is: the K
          // tile is then taken unread.
          if (!k_ready && !(ok = wait_k())) break;
          mma_commit_w(k_empty(kc % C::kKStages));
          ++kc;
        }
      }
    }
    // No MMA may still be running when TMEM is released.
    mma_commit_w(mma_done);
    mbar_wait_drain(mma_done, 0, args.wait_budget);
    __syncwarp();
  } else if (warp == kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    // ================================================================ TMA producer
    const int per_log = 7 - args.page_shift, per = 1 << per_log;   // pages per key tile
    const uint32_t page_bytes = static_cast<uint32_t>(D) << args.page_shift;
    uint32_t kn = 0, vn = 0;              // K and V tiles asked for so far
    Walker walk(args, pre, j0, j1);
    Seg s{};
    bool ok = true;
    while (ok && walk.next(s)) {
      Window cur, nxt;
      cur.load(args, s, s.a << per_log);
      nxt.load(args, s, cur.base + 32);
      for (int j = s.a; j < s.e; ++j) {
        if ((j << per_log) >= cur.base + 32) {
          cur = nxt;
          nxt.load(args, s, cur.base + 32);
        }
        int pid[4];
        uint32_t mask = 0u, bytes = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pid[i] = -1;
          if (i < per) {
            pid[i] = __shfl_sync(0xffffffffu, cur.pid, (j << per_log) + i - cur.base);
            if (pid[i] >= 0) {
              mask |= ((1u << (4 >> per_log)) - 1u) << (i * (4 >> per_log));
              bytes += page_bytes;
            }
          }
        }
        const uint32_t ks = kn % C::kKStages, vs = vn % C::kVStages;
        if (kn >= C::kKStages &&
            !mbar_wait_warp(k_empty(ks), (kn / C::kKStages - 1) & 1, wc, kWaitKvEmpty)) {
          ok = false;
          break;
        }
        const uint32_t kd = sbase + C::kKOff + ks * C::kCodeTile;
        mbar_arrive_expect_tx_w(k_full(ks), bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (pid[i] >= 0)
            tma_load_3d_w(kd + i * page_bytes, &tm_k, k_full(ks), 0, s.head << args.page_shift, pid[i]);
        ++kn;
        if (vn >= C::kVStages &&
            !mbar_wait_warp(v_empty(vs), (vn / C::kVStages - 1) & 1, wc, kWaitKvEmpty)) {
          ok = false;
          break;
        }
        const uint32_t vd = sbase + C::kVOff + vs * C::kCodeTile;
        if (lane == 0) valid[vs] = mask;
        __syncwarp();
        mbar_arrive_expect_tx_w(v_full(vs), bytes);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (pid[i] >= 0)
            tma_load_3d_w(vd + i * page_bytes, &tm_v, v_full(vs), 0, s.head << args.page_shift, pid[i]);
        ++vn;
      }
    }
    if (lane == 0) {
      // What is to be joined: the unit that this CTA starts and others go on
      // with (its last one).
      const bool shared_unit = ok && j1 > j0 && s.starts && !s.ends;
      args.rec[2 * cta] = shared_unit ? make_int4(s.r0, s.n, s.rb, s.head) : make_int4(0, 0, 0, 0);
      if (shared_unit)
        args.rec[2 * cta + 1] = make_int4(cta_of(W, G, j1 - (s.e - s.a) + s.nt - 1),
                                          static_cast<int>(W), static_cast<int>(W >> 32), 0);
    }
    // Every copy this warp started must have landed before the CTA exits.
    for (uint32_t r = kn > C::kKStages ? kn - C::kKStages : 0; r < kn; ++r)
      mbar_wait_drain(k_full(r % C::kKStages), (r / C::kKStages) & 1, args.wait_budget);
    for (uint32_t r = vn > C::kVStages ? vn - C::kVStages : 0; r < vn; ++r)
      mbar_wait_drain(v_full(r % C::kVStages), (r / C::kVStages) & 1, args.wait_budget);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    // ================================================================ V to fp16
    // The fp16 tile is laid out as the P V product reads it: two chunks of 64
    // columns, rows of 128 bytes with the 128-byte swizzle.  A thread takes
    // one 16-byte chunk of codes (16 columns) of a row at a time, eight
    // neighbouring lanes two rows of four, so that their stores meet
    // different banks.
    constexpr int CH = D / 16;            // 16-byte chunks of a code row
    constexpr int kIter = kBN * CH / 64;
    const int ct = tid - 32 * 10;         // 0 .. 63
    auto row_of = [](int id) { return D == 128 ? (id >> 4) * 2 + (id >> 2 & 1) : id >> 2; };
    auto chunk_of = [](int id) { return D == 128 ? (id & 3) | (id >> 3 & 1) << 2 : id & 3; };
    uint32_t cnt = 0;
    Walker walk(args, pre, j0, j1);
    Seg s;
    bool ok = true;
    while (ok && walk.next(s)) {
      for (int j = s.a; j < s.e; ++j) {
        const uint32_t st = cnt % C::kVStages, hs = cnt & 1;
        if (!mbar_wait_warp(v_full(st), (cnt / C::kVStages) & 1, wc, kWaitKvFull) ||
            (cnt > 1 && !mbar_wait_warp(h_empty(hs), ((cnt >> 1) - 1) & 1, wc, kWaitMmaDone))) {
          ok = false;
          break;
        }
        const uint32_t src = sbase + C::kVOff + st * C::kCodeTile;
        const uint32_t dst = sbase + C::kHOff + hs * C::kHalfTile;
        const uint32_t mask = valid[st];
        const int left = s.len - j * kBN;          // keys of the tile that exist
        const bool edge = left < kBN || mask != 0xfu;
#pragma unroll
        for (int i0 = 0; i0 < kIter; i0 += 4) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int id = ct + 64 * (i0 + i), row = row_of(id), c = chunk_of(id);
            w[i] = ld_shared_v4(src + code_off<D>(row, c));
            // Slots behind the end and pages that were not loaded hold
            // anything, NaN codes too.
            if (edge && (row >= left || !(mask >> (row >> 5) & 1u))) w[i] = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int id = ct + 64 * (i0 + i), row = row_of(id), c = chunk_of(id);
            const uint32_t base = dst + (c >> 2) * C::kHalfChunk + row * 128;
            const int c2 = 2 * (c & 3);            // 16-byte chunk of the fp16 row
            st_shared_v4(base + ((c2 ^ (row & 7)) << 4), e4m3x2_to_f16x2(w[i].x),
                         e4m3x2_to_f16x2(w[i].x >> 16), e4m3x2_to_f16x2(w[i].y),
                         e4m3x2_to_f16x2(w[i].y >> 16));
            st_shared_v4(base + (((c2 + 1) ^ (row & 7)) << 4), e4m3x2_to_f16x2(w[i].z),
                         e4m3x2_to_f16x2(w[i].z >> 16), e4m3x2_to_f16x2(w[i].w),
                         e4m3x2_to_f16x2(w[i].w >> 16));
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
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const CacheAttnArgs& a,
                     cudaStream_t stream) {
  auto kern = chunk_kernel<D>;
  const int smem = ChunkCfg<D>::kSmemFixed + (a.s.B + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // The register split inside the kernel is only valid for this launch size.
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  kern<<<a.grid, kThreads, smem, stream>>>(tk, tv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_cache_join(D, kUnitRows, a, stream);
}

}  // namespace

cudaError_t launch_cache_chunk(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CacheAttnArgs& a, cudaStream_t stream) {
  return d == 64 ? launch_t<64>(tk, tv, a, stream) : launch_t<128>(tk, tv, a, stream);
}

}  // namespace fattn
