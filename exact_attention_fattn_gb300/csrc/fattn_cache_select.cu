// Page selection for sparse attention over the paged 8-bit cache: for each
// new token and kv head, the pages whose keys may score highest.
//
// Score of a page: an upper bound of the sum of q . k over the head's group
// of queries, from the page's bounds lo <= k <= hi (int8):
//   sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d A+_d hi_d + A-_d lo_d,
//   A+ = sum_h max(q_h, 0), A- = sum_h min(q_h, 0),
// with q rounded to whole numbers of 1/127 of the group's largest entry.
// A+, A- <= 127 * 128 fit 16 bits and the sum stays below 2^31, so it is exact
// in any order, and with the page's power-of-two scale two programs that
// follow the definition choose the same pages.  Ties go to the lower page.
//
// Bound: the bounds' bytes, 2 d a page and head, streamed 16 bytes a lane with 8
// pages in flight per group of lanes, against 16 x 8 bit dot products, and latency
// where the pages are few.  The choice is a radix select, eight bits of the scores
// at a time.  A cluster of up to 8 CTAs scores and chooses for one (row, head) pair,
// scores in the first one's shared memory; where they do not fit there (10000
// pages), CTAs of 128 or 256 pages each score into the workspace and a second
// kernel chooses.  Measured: one row of 12 pairs on 938 pages, with the attention, 21.2
// us (23.6 without clusters).
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kSelThreads = 256;
constexpr int kOnceThreads = 512;
constexpr int kFewThreads = 128;
constexpr int kInFlight = 8;         // pages in flight per lane group
constexpr int kOncePages = 10000;    // scores that fit the 48 KB every kernel may use

// Position of a call's row; false when the row belongs to no sequence.
__device__ __forceinline__ bool row_position(const CacheSelectArgs& a, int row, int& b, int& pos) {
  b = find_last_warp(a.s.B, row, [&](int i) { return __ldg(a.s.q_start + i); });
  const SeqInfo q = seq_info(a.s, b, a.page_shift);
  if (!q.ok) {
    if (threadIdx.x == 0) record_bad_index(a.status, kSiteSeqStart);
    return false;
  }
  if (row < q.r0 || row >= q.r0 + q.n) return false;
  pos = q.len - q.n + (row - q.r0);
  return true;
}

// 16 bytes that are read once, in program order with other such loads (the
// compiler otherwise waits for one before it asks for the next).
__device__ __forceinline__ int4 ld_stream(const int8_t* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Cluster barrier, and a store to the shared memory of a cluster's first CTA.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t first_cta_addr(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

// The group's query sums A- and A+ of a row and head, and from them the
// scores of pages, by all NT threads of a CTA.
template <int D, int NT>
struct Scorer {
  static constexpr int LP = 2 * D / 16;                // lanes per page: 16 bytes each
  static constexpr int kGroups = NT / LP;
  static constexpr int kPages = kGroups * kInFlight;   // pages at a time
  static constexpr int kParts = NT / D;
  struct Shared {
    float red[NT / 32];
    int sums[2][kParts][D];
    alignas(16) int16_t avec[2][D];                    // A- (meets lo), A+ (meets hi)
  };
  const CacheSelectArgs& a;
  const int head, b;
  int av[8];                                           // this lane's 16 columns of one of them

  __device__ __forceinline__ Scorer(const CacheSelectArgs& args, Shared& sh, int row, int h, int seq)
      : a(args), head(h), b(seq) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tid % D, part = tid / D;
    const uint16_t* qp = a.q + row * a.q_row + static_cast<long long>(head) * a.group * D + col;
    float amax = 0.f;
    for (int g = part; g < a.group; g += kParts)
      amax = fmaxf(amax, fabsf(__uint_as_float(static_cast<uint32_t>(__ldg(qp + g * D)) << 16)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (lane == 0) sh.red[warp] = amax;
    __syncthreads();
    amax = sh.red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) amax = fmaxf(amax, sh.red[w]);
    // Queries below 2^-100 count as zero (127 / amax would overflow).
    const float inv = amax >= 7.888609052210118e-31f ? __fdiv_rn(127.f, amax) : 0.f;
    int up = 0, down = 0;
    for (int g = part; g < a.group; g += kParts) {
      const float x = __uint_as_float(static_cast<uint32_t>(__ldg(qp + g * D)) << 16);
      const int v = max(-127, min(127, __float2int_rn(__fmul_rn(x, inv))));
      up += max(v, 0);
      down += min(v, 0);
    }
    sh.sums[0][part][col] = down;
    sh.sums[1][part][col] = up;
    __syncthreads();
    for (int i = tid; i < 2 * D; i += NT) {
      int t = 0;
#pragma unroll
      for (int q = 0; q < kParts; ++q) t += sh.sums[i / D][q][i % D];
      sh.avec[i / D][i % D] = static_cast<int16_t>(t);
    }
    __syncthreads();
    const int gl = tid % LP;
    const int4* p = reinterpret_cast<const int4*>(&sh.avec[gl / (LP / 2)][(gl % (LP / 2)) * 16]);
    const int4 x = p[0], y = p[1];
    av[0] = x.x; av[1] = x.y; av[2] = x.z; av[3] = x.w;
    av[4] = y.x; av[5] = y.y; av[6] = y.z; av[7] = y.w;
  }

  // Lane i < kInFlight of a group looks page i of the group's up.
  struct Pages {
    int mine, pid;
    float ks;
  };
  __device__ __forceinline__ Pages look_up(int p0, int n) const {
    const int gl = threadIdx.x % LP, group = threadIdx.x / LP;
    Pages r{p0 + group + (gl & (kInFlight - 1)) * kGroups, -1, 0.f};
    if (gl < kInFlight && r.mine < n) {
      r.pid = __ldg(a.s.table + static_cast<long long>(b) * a.s.max_pages + r.mine);
      if (r.pid < 0 || r.pid >= a.pages) {
        record_bad_index(a.status, kSitePage);
        r.pid = -1;
      } else {
        r.ks = __ldg(a.k_scale + static_cast<long long>(r.pid) * a.Hkv + head);
      }
    }
    return r;
  }
  // Scores of the pages looked up, as out(page, score); -inf for a page that is
  // not there.
  template <class Out>
  __device__ __forceinline__ void score(const Pages& r, int n, Out out) const {
    const int gl = threadIdx.x % LP, src0 = (threadIdx.x & 31) & ~(LP - 1);
    int4 w[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      // a page that is not there: page 0 is read and not used, so that the
      // loads go out together
      const int id = max(0, __shfl_sync(0xffffffffu, r.pid, src0 + i));
      w[i] = ld_stream(a.bounds + (static_cast<long long>(id) * a.Hkv + head) * 2 * D + 16 * gl);
    }
    int mine_sum = 0;
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      int s = __dp2a_lo(av[0], w[i].x, 0);
      s = __dp2a_hi(av[1], w[i].x, s);
      s = __dp2a_lo(av[2], w[i].y, s);
      s = __dp2a_hi(av[3], w[i].y, s);
      s = __dp2a_lo(av[4], w[i].z, s);
      s = __dp2a_hi(av[5], w[i].z, s);
      s = __dp2a_lo(av[6], w[i].w, s);
      s = __dp2a_hi(av[7], w[i].w, s);
#pragma unroll
      for (int off = LP / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (gl == i) mine_sum = s;
    }
    if (gl < kInFlight && r.mine < n && dcheck(inside(r.mine, 1, a.s.max_pages), a.status, 611))
      out(r.mine, r.pid >= 0 ? __fmul_rn(__int2float_rn(mine_sum), r.ks) : -INFINITY);
  }
};

// Scores in an order that unsigned comparison keeps; forced pages on top.
__device__ __forceinline__ uint32_t order_key(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct ChooseShared {
  int hist[256];
  int wsum[2][32];
  uint32_t prefix;
  int left;
};

// The k highest of n > k scores (shared or global memory), ascending, to out.
template <int NT>
__device__ __forceinline__ void choose(const CacheSelectArgs& a, ChooseShared& sh, const float* sc, int n,
                                       int* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int k = a.n_selected;
  auto key_of = [&](int i) -> uint32_t {
    return (i < a.n_first || i >= n - a.n_recent) ? 0xffffffffu : order_key(sc[i]);
  };
  // The k-th highest key, eight bits at a time: among the keys that share the
  // prefix found so far, `left` are still to be taken.
  uint32_t prefix = 0u;
  int left = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += NT) sh.hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : (0xffffffffu << (shift + 8));
    for (int i = tid; i < n; i += NT) {
      const uint32_t key = key_of(i);
      if ((key & above) == prefix) atomicAdd(&sh.hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l, highest first
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = sh.hist[255 - 8 * lane - i];
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
      }
      int before = incl - sum;
      if (before < left && incl >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < left && before + c[i] >= left) {
            sh.prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
            sh.left = left - before;
            break;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    prefix = sh.prefix;
    left = sh.left;
  }
  // All keys above the threshold, and the first `left` equal to it, in order.
  int done = 0, ties = 0;
  for (int i0 = 0; i0 < n; i0 += NT) {
    const int i = i0 + tid;
    const uint32_t key = i < n ? key_of(i) : 0u;
    const bool gt = i < n && key > prefix, eq = i < n && key == prefix;
    const unsigned int meq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) sh.wsum[0][warp] = __popc(meq);
    __syncthreads();
    int tie = ties + __popc(meq & ((1u << lane) - 1u)), all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) tie += sh.wsum[0][w];
      all += sh.wsum[0][w];
    }
    ties += all;
    const bool take = gt || (eq && tie < left);
    const unsigned int mt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) sh.wsum[1][warp] = __popc(mt);
    __syncthreads();
    int slot = done + __popc(mt & ((1u << lane) - 1u));
    all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) slot += sh.wsum[1][w];
      all += sh.wsum[1][w];
    }
    done += all;
    if (take && slot < k && dcheck(inside(slot, 1, k) && inside(i, 1, n), a.status, 614)) out[slot] = i;
  }
}

// Pages up to a row's own; where they are no more than are wanted, all are taken.
__device__ __forceinline__ bool take_all(const CacheSelectArgs& a, int n, int* out) {
  if (n > a.n_selected) return false;
  for (int i = threadIdx.x; i < a.n_selected; i += blockDim.x) out[i] = i < n ? i : -1;
  return true;
}

// Grid (T + 1, Hkv, C) in clusters of C along z: the cluster's CTAs score 1 / C of a
// pair's pages each, into the first one's shared memory, and that one chooses.
// The last row's CTAs check the batch.
template <int D, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) select_kernel(const __grid_constant__ CacheSelectArgs a) {
  using S = Scorer<D, NT>;
  __shared__ union {
    typename S::Shared score;
    ChooseShared choose;
  } sh;
  extern __shared__ float scores[];
  const int row = blockIdx.x, head = blockIdx.y, rank = blockIdx.z;
  const bool shared = gridDim.z > 1;
  if (row == a.s.T) {                  // CTAs of their own (beside a pair's scores it cost 1.5 us of 22)
    if (head == 0 && rank == 0) check_seqs(a.s, threadIdx.x, NT, a.page_shift, a.status);
    return;
  }
  if (shared) cluster_arrive();        // the first CTA has started when others write to it
  int b, pos;
  // the same for all CTAs of a cluster
  if (!row_position(a, row, b, pos)) return;
  const int n = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
  int* out = a.selected + (static_cast<long long>(row) * a.Hkv + head) * a.n_selected;
  if (!dcheck(row < a.s.T && head < a.Hkv && n <= a.s.max_pages, a.status, 615)) return;
  if (n <= a.n_selected) {
    if (rank == 0) take_all(a, n, out);
    return;
  }
  const int p1 = rank * S::kPages, step = gridDim.z * S::kPages;
  const S s(a, sh.score, row, head, b);
  typename S::Pages next = s.look_up(p1, n);
  const uint32_t to = first_cta_addr(smem_u32(scores));
  if (shared) cluster_wait();
  for (int p0 = p1; p0 < n; p0 += step) {
    const typename S::Pages cur = next;
    if (p0 + step < n) next = s.look_up(p0 + step, n);
    s.score(cur, n, [&](int page, float x) {
      if (dcheck(inside(4 * page, 4, dynamic_smem_bytes()), a.status, 612)) st_cluster(to + 4 * page, x);
    });
  }
  if (shared) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
  }
  __syncthreads();
  choose<NT>(a, sh.choose, scores, n, out);
}

// Grid (T, Hkv, chunks of pages): scores to the workspace.
template <int D>
__global__ void __launch_bounds__(kSelThreads, 4) score_kernel(const __grid_constant__ CacheSelectArgs a) {
  using S = Scorer<D, kSelThreads>;
  __shared__ typename S::Shared sh;
  allow_child();
  const int row = blockIdx.x, head = blockIdx.y, p0 = blockIdx.z * S::kPages;
  int b, pos;
  if (!row_position(a, row, b, pos)) return;
  const int n = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
  if (p0 >= n || n <= a.n_selected) return;   // few pages: all are taken
  const S s(a, sh, row, head, b);
  const long long at = (static_cast<long long>(row) * a.Hkv + head) * a.s.max_pages;
  if (!dcheck(inside(at, n, static_cast<long long>(a.s.T) * a.Hkv * a.s.max_pages), a.status, 613)) return;
  float* out = a.scores + at;
  s.score(s.look_up(p0, n), n, [&](int page, float x) { out[page] = x; });
}

// Grid (T, Hkv): choice from the workspace.
__global__ void __launch_bounds__(kSelThreads, 4) choose_kernel(const __grid_constant__ CacheSelectArgs a) {
  __shared__ ChooseShared sh;
  const int row = blockIdx.x, head = blockIdx.y;
  if (row == 0 && head == 0) check_seqs(a.s, threadIdx.x, kSelThreads, a.page_shift, a.status);
  wait_for_parent();
  int b, pos;
  if (!row_position(a, row, b, pos)) return;
  const int n = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
  const long long at = static_cast<long long>(row) * a.Hkv + head;
  int* out = a.selected + at * a.n_selected;
  if (take_all(a, n, out)) return;
  choose<kSelThreads>(a, sh, a.scores + at * a.s.max_pages, n, out);
}

template <int D, int NT>
cudaError_t launch_once(const CacheSelectArgs& a, unsigned ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = ctas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.s.T) + 1u, a.Hkv, ctas);
  cfg.blockDim = NT;
  cfg.dynamicSmemBytes = a.s.max_pages * sizeof(float);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<D, NT>, a);
}

template <int D>
cudaError_t launch_t(const CacheSelectArgs& a, cudaStream_t stream) {
  const dim3 pairs(a.s.T, a.Hkv);
  if (cache_select_at_once(a.s.max_pages)) {
    // Many pairs, or few pages: CTAs of 128 threads, eight to an SM, as a pair's
    // time is mostly latency.  Measured with the attention over 5 pages (d = 128,
    // 128 / 512 threads, us): 384 pairs, 100 pages 24.8 / 33.2, 400 pages 33.6 /
    // 36.8; 1536 pairs, 24 pages 51 / 87, 400 pages 81 / 93; 160 pairs, 100 pages
    // 20.5 / 21.9, but 400 pages 26.7 / 23.5.
    const long long n_pairs = static_cast<long long>(a.s.T) * a.Hkv;
    if (n_pairs > 2 * kSms || a.s.max_pages <= 2 * Scorer<D, kFewThreads>::kPages)
      return launch_once<D, kFewThreads>(a, 1, stream);
    // Otherwise as many CTAs per pair as have pages and fit the GPU beside the others.
    constexpr int kPages = Scorer<D, kOnceThreads>::kPages;
    unsigned ctas = 1;
    while (ctas < 8 && ctas * n_pairs <= kSms && static_cast<int>(ctas) * kPages < a.s.max_pages) ctas *= 2;
    return launch_once<D, kOnceThreads>(a, ctas, stream);
  }
  constexpr int kPages = Scorer<D, kSelThreads>::kPages;
  score_kernel<D><<<dim3(a.s.T, a.Hkv, (a.s.max_pages + kPages - 1) / kPages), kSelThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_child(choose_kernel, pairs, kSelThreads, 0, stream, a);
}

}  // namespace

// One kernel as long as a pair's scores fit one CTA's shared memory.  Measured
// with the attention over 16 selected pages of 64, 8 kv heads, d = 128 (one kernel
// in clusters / without clusters / two kernels, us): 1 row, 2048 pages 21.8 / 28 /
// 27.4; 1 row, 8000 pages 35 / 64 / 45; 4 rows, 4000 pages 34 / - / 42; 16 rows, 2000
// pages 43 in each way.
bool cache_select_at_once(int max_pages) { return max_pages <= kOncePages; }

cudaError_t launch_cache_select(int d, const CacheSelectArgs& a, cudaStream_t stream) {
  return d == 64 ? launch_t<64>(a, stream) : launch_t<128>(a, stream);
}

}  // namespace fattn
