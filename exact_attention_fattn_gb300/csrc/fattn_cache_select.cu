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
// Bound: the bounds' bytes, 2 d a page and head.  The score kernel streams
// them, 16 bytes a lane and 8 pages in flight per group of lanes, with 16 x 8
// bit dot products; the choice is a radix select over the scores, which are
// in L2 by then, 4 bytes each.
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kSelThreads = 256;
constexpr int kInFlight = 8;         // pages in flight per lane group

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

// Grid (T, Hkv, chunks of pages).
template <int D>
__global__ void __launch_bounds__(kSelThreads) score_kernel(const CacheSelectArgs a) {
  constexpr int LP = 2 * D / 16;                       // lanes per page: 16 bytes each
  constexpr int kGroups = kSelThreads / LP;
  constexpr int kPages = kGroups * kInFlight;          // pages per CTA
  constexpr int kParts = kSelThreads / D;
  __shared__ float red[kSelThreads / 32];
  __shared__ int sums[2][kParts][D];
  __shared__ __align__(16) int16_t avec[2][D];         // A- (meets lo), A+ (meets hi)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, head = blockIdx.y;
  int b, pos;
  if (!row_position(a, row, b, pos)) return;
  const int n_pages = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
  const int p0 = blockIdx.z * kPages;
  if (p0 >= n_pages || n_pages <= a.n_selected) return;   // few pages: all are taken

  // ---- the group's query sums
  const int col = tid % D, part = tid / D;
  const uint16_t* qp = a.q + row * a.q_row + static_cast<long long>(head) * a.group * D + col;
  float amax = 0.f;
  for (int h = part; h < a.group; h += kParts)
    amax = fmaxf(amax, fabsf(__uint_as_float(static_cast<uint32_t>(__ldg(qp + h * D)) << 16)));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < kSelThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  // Queries below 2^-100 count as zero (127 / amax would overflow).
  const float inv = amax >= 7.888609052210118e-31f ? __fdiv_rn(127.f, amax) : 0.f;
  int up = 0, down = 0;
  for (int h = part; h < a.group; h += kParts) {
    const float x = __uint_as_float(static_cast<uint32_t>(__ldg(qp + h * D)) << 16);
    const int v = max(-127, min(127, __float2int_rn(__fmul_rn(x, inv))));
    up += max(v, 0);
    down += min(v, 0);
  }
  sums[0][part][col] = down;
  sums[1][part][col] = up;
  __syncthreads();
  for (int i = tid; i < 2 * D; i += kSelThreads) {
    int t = 0;
#pragma unroll
    for (int q = 0; q < kParts; ++q) t += sums[i / D][q][i % D];
    avec[i / D][i % D] = static_cast<int16_t>(t);
  }
  __syncthreads();

  // ---- this lane's 16 columns of lo (first half of the group) or hi
  const int gl = tid % LP, group = tid / LP;
  const int side = gl / (LP / 2), c0 = (gl % (LP / 2)) * 16;
  int av[8];
  {
    const int4* p = reinterpret_cast<const int4*>(&avec[side][c0]);
    const int4 x = p[0], y = p[1];
    av[0] = x.x; av[1] = x.y; av[2] = x.z; av[3] = x.w;
    av[4] = y.x; av[5] = y.y; av[6] = y.z; av[7] = y.w;
  }
  // Lane i < kInFlight of a group looks page i of the group up.
  const int src0 = lane & ~(LP - 1);
  int pid = -1;
  float ks = 0.f;
  const int mine = p0 + group + (gl & (kInFlight - 1)) * kGroups;
  if (gl < kInFlight && mine < n_pages) {
    pid = __ldg(a.s.table + static_cast<long long>(b) * a.s.max_pages + mine);
    if (pid < 0 || pid >= a.pages) {
      record_bad_index(a.status, kSitePage);
      pid = -1;
    } else {
      ks = __ldg(a.k_scale + static_cast<long long>(pid) * a.Hkv + head);
    }
  }
  int4 w[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    const int id = __shfl_sync(0xffffffffu, pid, src0 + i);
    w[i] = make_int4(0, 0, 0, 0);
    if (id >= 0)
      w[i] = __ldg(reinterpret_cast<const int4*>(
          a.bounds + (static_cast<long long>(id) * a.Hkv + head) * 2 * D + 16 * gl));
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
  if (gl < kInFlight && mine < n_pages)
    a.scores[(static_cast<long long>(row) * a.Hkv + head) * a.s.max_pages + mine] =
        pid >= 0 ? __fmul_rn(__int2float_rn(mine_sum), ks) : -INFINITY;
}

// Scores in an order that unsigned comparison keeps; forced pages on top.
__device__ __forceinline__ uint32_t order_key(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Grid (T, Hkv): the n_selected highest of a row's scores, ascending.
__global__ void __launch_bounds__(kSelThreads) choose_kernel(const CacheSelectArgs a) {
  __shared__ int hist[256];
  __shared__ int wsum[2][kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, head = blockIdx.y;
  int b, pos;
  if (!row_position(a, row, b, pos)) return;
  const int n = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
  const long long at = static_cast<long long>(row) * a.Hkv + head;
  int* out = a.selected + at * a.n_selected;
  const int k = a.n_selected;
  if (n <= k) {
    for (int i = tid; i < k; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const float* sc = a.scores + at * a.s.max_pages;
  auto key_of = [&](int i) -> uint32_t {
    return (i < a.n_first || i >= n - a.n_recent) ? 0xffffffffu : order_key(sc[i]);
  };
  // The k-th highest key, eight bits at a time: among the keys that share the
  // prefix found so far, `left` are still to be taken.
  uint32_t prefix = 0u;
  int left = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : (0xffffffffu << (shift + 8));
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t key = key_of(i);
      if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l, highest first
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
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
            s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
            s_left = left - before;
            break;
          }
          before += c[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // All keys above the threshold, and the first `left` equal to it, in order.
  int done = 0, ties = 0;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const uint32_t key = i < n ? key_of(i) : 0u;
    const bool gt = i < n && key > prefix, eq = i < n && key == prefix;
    const unsigned int meq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) wsum[0][warp] = __popc(meq);
    __syncthreads();
    int tie = ties + __popc(meq & ((1u << lane) - 1u)), all = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) tie += wsum[0][w];
      all += wsum[0][w];
    }
    ties += all;
    const bool take = gt || (eq && tie < left);
    const unsigned int mt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) wsum[1][warp] = __popc(mt);
    __syncthreads();
    int slot = done + __popc(mt & ((1u << lane) - 1u));
    all = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) slot += wsum[1][w];
      all += wsum[1][w];
    }
    done += all;
    if (take && slot < k) out[slot] = i;
  }
}

template <int D>
cudaError_t launch_t(const CacheSelectArgs& a, cudaStream_t stream) {
  constexpr int kPages = kSelThreads / (2 * D / 16) * kInFlight;
  if (a.s.max_pages > a.n_selected) {
    const dim3 grid(a.s.T, a.Hkv, (a.s.max_pages + kPages - 1) / kPages);
    score_kernel<D><<<grid, kSelThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  choose_kernel<<<dim3(a.s.T, a.Hkv), kSelThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_select(int d, const CacheSelectArgs& a, cudaStream_t stream) {
  return d == 64 ? launch_t<64>(a, stream) : launch_t<128>(a, stream);
}

}  // namespace fattn
