// Appending to the paged 8-bit cache: new keys (rotated by their positions)
// and values are quantised to e4m3 with one power-of-two scale per page and
// head, and new queries are rotated on the way.
//
// A page of a head has scale 2^e with e the smallest exponent that holds its
// tokens, amax <= 448 * 2^e.  A new token may raise e; the page's earlier
// codes are then multiplied by 2^(e_old - e) and rounded again.  With scales
// that are powers of two this changes nothing but codes that become
// subnormal, and a value's precision does not depend on which neighbour
// raised the scale; scales amax / 448 would round every earlier code afresh at
// each raise.  A page whose first token is among the new ones starts over.
//
// The rotation takes its cosines and sines from a table in fp32; products and
// sums are rounded one by one (no fused multiply-add), so the codes do not
// depend on how a compiler contracts them.
//
// Bound: the bytes of q, k, v in and q, codes out.  A CTA of 128 threads takes one
// page of one head, K and V together, 8 or 16 tokens at a time; where the page gets more, the
// maximum and the quantisation are two passes, the second out of L1 and L2.
// Further CTAs rotate q, eight heads of a token per thread, whose cosines and
// sines are the same.  Eight CTAs per SM (64 registers) and two turns of the
// first pass in flight took four prompts of 4096 tokens (32 query and 8 kv
// heads, d = 128) from 88 to 72 us, 68 % of the bytes' time; single tokens of 32
// sequences take 6.9 us, all latency.  CTAs that held a whole page in
// registers instead (up to 1024 threads) were slower at both ends: 96 and 10.3 us.
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kQHeads = 8;            // query heads per thread
constexpr int kThreads = 128;

__device__ __forceinline__ void bf16x8_to_f32(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Cosines and sines of the 8 columns [8 cc, 8 cc + 8) of a row: of its 8
// columns where halves pair, of its 4 pairs where neighbours do.  cs: the
// row's table entry, or nullptr where there is no row.
struct Angles {
  float4 c[2], s[2];
  bool in;            // whether the columns are rotated
  bool low;           // halves: in the first half
  __device__ __forceinline__ Angles(const float* cs, int rope_dim, int interleaved, int cc) {
    const int h = rope_dim >> 1, dim = 8 * cc;
    in = cs != nullptr && dim < rope_dim;
    low = dim < h;
    if (!in) return;
    const int at = interleaved ? dim >> 1 : (low ? dim : dim - h);
    c[0] = __ldg(reinterpret_cast<const float4*>(cs + at));
    s[0] = __ldg(reinterpret_cast<const float4*>(cs + h + at));
    if (interleaved) return;
    c[1] = __ldg(reinterpret_cast<const float4*>(cs + at + 4));
    s[1] = __ldg(reinterpret_cast<const float4*>(cs + h + at + 4));
  }
};

// Rotates 8 columns of a row that CH = D / 8 neighbouring lanes hold; every
// lane of the warp takes part.
template <int CH>
__device__ __forceinline__ void rotate8(const uint4& w, float (&f)[8], const Angles& a, int rope_dim,
                                        int interleaved, int cc) {
  bf16x8_to_f32(w, f);
  if (rope_dim == 0) return;   // the same for the whole launch
  if (interleaved) {
    if (!a.in) return;
    const float cv[4] = {a.c[0].x, a.c[0].y, a.c[0].z, a.c[0].w};
    const float sv[4] = {a.s[0].x, a.s[0].y, a.s[0].z, a.s[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[2 * i], y = f[2 * i + 1];
      f[2 * i] = __fsub_rn(__fmul_rn(x, cv[i]), __fmul_rn(y, sv[i]));
      f[2 * i + 1] = __fadd_rn(__fmul_rn(y, cv[i]), __fmul_rn(x, sv[i]));
    }
    return;
  }
  // halves: column i pairs with column i + h, h / 8 chunks away
  const int hc = rope_dim >> 4;
  const int pc = 8 * cc < rope_dim ? (cc < hc ? cc + hc : cc - hc) : cc;
  const int src = ((threadIdx.x & 31) & ~(CH - 1)) | pc;
  uint4 p;
  p.x = __shfl_sync(0xffffffffu, w.x, src);
  p.y = __shfl_sync(0xffffffffu, w.y, src);
  p.z = __shfl_sync(0xffffffffu, w.z, src);
  p.w = __shfl_sync(0xffffffffu, w.w, src);
  if (!a.in) return;
  float g[8];
  bf16x8_to_f32(p, g);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float cv[4] = {a.c[q].x, a.c[q].y, a.c[q].z, a.c[q].w};
    const float sv[4] = {a.s[q].x, a.s[q].y, a.s[q].z, a.s[q].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = __fmul_rn(f[4 * q + i], cv[i]), y = __fmul_rn(g[4 * q + i], sv[i]);
      f[4 * q + i] = a.low ? __fsub_rn(x, y) : __fadd_rn(x, y);
    }
  }
}

// The smallest e in [kScaleExpMin, kScaleExpMax] with amax <= 448 * 2^e
// (448 = 1.75 * 2^8, the mantissa field of 1.75 is 0x600000).
__device__ __forceinline__ int amax_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kScaleExpMin, min(kScaleExpMax, e));
}

__device__ __forceinline__ uint2 encode8(const float (&f)[8], float mul) {
  uint2 c;
  c.x = pack_e4m3x4(__fmul_rn(f[0], mul), __fmul_rn(f[1], mul), __fmul_rn(f[2], mul),
                    __fmul_rn(f[3], mul));
  c.y = pack_e4m3x4(__fmul_rn(f[4], mul), __fmul_rn(f[5], mul), __fmul_rn(f[6], mul),
                    __fmul_rn(f[7], mul));
  return c;
}

__device__ __forceinline__ uint32_t rescale4(uint32_t w, float mul) {
  const float4 x = e4m3x4_to_f32x4(w);
  return pack_e4m3x4(__fmul_rn(x.x, mul), __fmul_rn(x.y, mul), __fmul_rn(x.z, mul),
                     __fmul_rn(x.w, mul));
}

// Bounds of the codes are kept in units of 448 / 127 of the scale.
__device__ __forceinline__ float bound_units(float code) {
  return __fdiv_rn(__fmul_rn(code, 127.f), 448.f);
}

// The codes of a head's page that were there before, times 2^(e_old - e).
template <int D, int NT>
__device__ __forceinline__ void rescale_rows(uint8_t* base, int rows, float mul) {
  uint4* p = reinterpret_cast<uint4*>(base);
  for (int i = threadIdx.x; i < rows * (D / 16); i += NT) {
    uint4 w = p[i];
    w.x = rescale4(w.x, mul);
    w.y = rescale4(w.y, mul);
    w.z = rescale4(w.z, mul);
    w.w = rescale4(w.w, mul);
    p[i] = w;
  }
}

// Why nothing of a sequence is appended or rotated (0: all of it is).  Its queries
// and its keys are left out together.
__device__ __forceinline__ unsigned int append_fault(const CacheAppendArgs& a, const SeqInfo& q) {
  if (!q.ok) return kSiteSeqStart;
  if (q.n > 0 && (q.len < q.n || (a.rope_dim > 0 && q.len > a.rope_len))) return kSitePosition;
  return 0u;
}

// Queries: CH lanes take a token's columns, each for kQHeads heads, whose
// angles are the same.  Item = token * groups of heads + group; a block of NT threads has
// NT / CH items.
template <int D, int SHIFT>
__device__ __forceinline__ void rotate_q(const CacheAppendArgs& a, int item) {
  constexpr int CH = D / 8;
  const int cc = threadIdx.x % CH;
  const int groups = (a.Hq + kQHeads - 1) / kQHeads;
  const int row = item / groups, h0 = (item - row * groups) * kQHeads;
  const float* cs = nullptr;
  bool on = row < a.s.T;
  if (on) {
    // the token's sequence: a guess for sequences of equal rows, else a search
    int b = static_cast<int>(static_cast<long long>(row) * a.s.B / a.s.T);
    if (row < __ldg(a.s.q_start + b) || row >= __ldg(a.s.q_start + b + 1)) {
      b = 0;
      for (int hi = a.s.B; hi - b > 1;) {
        const int mid = (b + hi) >> 1;
        if (__ldg(a.s.q_start + mid) <= row) b = mid; else hi = mid;
      }
    }
    const SeqInfo q = seq_info(a.s, b, SHIFT);
    on = row >= q.r0 && row < q.r0 + q.n;    // else behind the last sequence, or of a senseless one
    const unsigned int site = append_fault(a, q);
    if (site != 0u) {
      record_bad_index(a.status, site);
      on = false;
    }
    const int pos = q.len - q.n + (row - q.r0);
    if (on && a.rope_dim > 0 && dcheck(inside(pos, 1, a.rope_len), a.status, 601))
      cs = a.rope + static_cast<long long>(pos) * a.rope_dim;
  }
  uint4 w[kQHeads];
#pragma unroll
  for (int i = 0; i < kQHeads; ++i) {
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (on && h0 + i < a.Hq)               // q_out may be q, so this is no read-only data
      w[i] = *reinterpret_cast<const uint4*>(a.q + row * a.q_row + (h0 + i) * D + 8 * cc);
  }
  const Angles ang(cs, a.rope_dim, a.interleaved, cc);
#pragma unroll
  for (int i = 0; i < kQHeads; ++i) {
    float f[8];
    rotate8<CH>(w[i], f, ang, a.rope_dim, a.interleaved, cc);
    if (on && h0 + i < a.Hq &&
        dcheck(inside((static_cast<long long>(row) * a.Hq + h0 + i) * D + 8 * cc, 8,
                      static_cast<long long>(a.s.T) * a.Hq * D), a.status, 602))
      *reinterpret_cast<uint4*>(a.q_out + (static_cast<long long>(row) * a.Hq + h0 + i) * D + 8 * cc) =
          make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7]));
  }
}

// The page's bounds from each thread's extremes of its 8 columns (of the codes
// it wrote), and, where the page goes on, the bounds it had, times 2^shift.
template <int D, int NT>
__device__ __forceinline__ void store_bounds(int8_t* out, float (&bnd)[2][NT / 32][D], float (&low)[8],
                                             float (&high)[8], bool goes_on, int shift) {
  constexpr int CH = D / 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cc = tid % CH;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = 16; off >= CH; off >>= 1) {
      low[i] = fminf(low[i], __shfl_xor_sync(0xffffffffu, low[i], off));
      high[i] = fmaxf(high[i], __shfl_xor_sync(0xffffffffu, high[i], off));
    }
    if (lane < CH) {
      bnd[0][warp][8 * cc + i] = low[i];
      bnd[1][warp][8 * cc + i] = high[i];
    }
  }
  __syncthreads();
  for (int at = tid; at < 2 * D; at += NT) {
    const int side = at / D, col = at % D;
    float x = bnd[side][0][col];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w)
      x = side ? fmaxf(x, bnd[side][w][col]) : fminf(x, bnd[side][w][col]);
    // rounded outwards: a page's bounds stay bounds
    if (isfinite(x)) x = side ? ceilf(bound_units(x)) : floorf(bound_units(x));
    if (goes_on) {
      const float old = __fmul_rn(static_cast<float>(out[at]), exp2i(shift));
      x = side ? fmaxf(x, ceilf(old)) : fminf(x, floorf(old));
    }
    if (!isfinite(x)) x = 0.f;   // a fresh page of NaN tokens alone
    out[at] = static_cast<int8_t>(x);
  }
}

// A page that receives tokens: slots [lo, hi) of the sequence's page p.
struct PageWork {
  SeqInfo q;
  int p, lo, hi;
  int pid;            // -1: none
};

// Work units of the new tokens' pages: sequence b's are numbered from
// q_start[b] / page + 2 b.  n tokens touch at most n / page + 2 pages, so the
// ranges hold them; units past a sequence's last page do nothing.  The whole
// block looks its unit up.
template <int SHIFT>
__device__ __forceinline__ PageWork find_page(const CacheAppendArgs& a, int u) {
  constexpr int PAGE = 1 << SHIFT;
  PageWork w;
  w.pid = -1;
  auto first_unit = [&](int i) { return (__ldg(a.s.q_start + i) >> SHIFT) + 2 * i; };
  const int b = find_last_warp(a.s.B, u, first_unit);
  w.q = seq_info(a.s, b, SHIFT);
  const unsigned int site = append_fault(a, w.q);
  if (site != 0u) {
    if (threadIdx.x == 0) record_bad_index(a.status, site);
    return w;
  }
  const int nth = u - first_unit(b);
  if (nth < 0 || w.q.n == 0) return w;
  const int pos0 = w.q.len - w.q.n;
  w.p = (pos0 >> SHIFT) + nth;
  if (w.p >= (w.q.len + PAGE - 1) >> SHIFT) return w;
  w.lo = max(pos0 - (w.p << SHIFT), 0);
  w.hi = min(w.q.len - (w.p << SHIFT), PAGE);
  const int pid = __ldg(a.s.table + static_cast<long long>(b) * a.s.max_pages + w.p);
  if (pid < 0 || pid >= a.pages) {
    if (threadIdx.x == 0) record_bad_index(a.status, kSitePage);
    return w;
  }
  w.pid = pid;
  return w;
}

template <int D, int SHIFT>
__global__ void __launch_bounds__(kThreads, 8) append_kernel(const __grid_constant__ CacheAppendArgs a,
                                                                 int units) {
  constexpr int NT = kThreads, CH = D / 8, PAGE = 1 << SHIFT, kRows = NT / CH;
  __shared__ float red[2][NT / 32];
  __shared__ float bnd[2][NT / 32][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cc = tid % CH, row = tid / CH;
  const long long kv_blocks = static_cast<long long>(units) * a.Hkv;
  if (blockIdx.x == gridDim.x - 1) {   // a block of its own: in a unit's it cost 1.3 us of 6.9
    check_seqs(a.s, tid, NT, SHIFT, a.status);
    return;
  }
  if (blockIdx.x >= kv_blocks) {
    rotate_q<D, SHIFT>(a, static_cast<int>(blockIdx.x - kv_blocks) * kRows + row);
    return;
  }
  const int u = blockIdx.x / a.Hkv, head = blockIdx.x - u * a.Hkv;
  const PageWork pw = find_page<SHIFT>(a, u);
  if (pw.pid < 0) return;
  const int lo = pw.lo, hi = pw.hi, pos0 = pw.q.len - pw.q.n;
  const long long sc = static_cast<long long>(pw.pid) * a.Hkv + head;
  const int ek_old = scale_exp(a.k_scale[sc]), ev_old = scale_exp(a.v_scale[sc]);
  uint8_t* kp = a.k + pw.pid * a.page_stride + static_cast<long long>(head) * PAGE * D;
  uint8_t* vp = a.v + pw.pid * a.page_stride + static_cast<long long>(head) * PAGE * D;
  // the head's page, its slots and their rows of the call
  if (!dcheck(inside(pw.pid * a.page_stride + static_cast<long long>(head) * PAGE * D, PAGE * D,
                     a.pages * a.page_stride) &&
                  inside(sc, 1, static_cast<long long>(a.pages) * a.Hkv) && lo >= 0 && lo < hi && hi <= PAGE &&
                  inside(pw.q.r0 + ((pw.p << SHIFT) + lo - pos0), hi - lo, a.s.T) &&
                  (a.rope_dim == 0 || inside((pw.p << SHIFT) + lo, hi - lo, a.rope_len)),
              a.status, 603))
    return;

  float kf[8], vf[8];
  bool nan_row = false;
  auto load = [&](int t) {               // slot t's key, rotated, and value
    const bool on = t < hi;
    uint4 w = make_uint4(0u, 0u, 0u, 0u), v = w;
    const float* cs = nullptr;
    if (on) {
      const long long src = pw.q.r0 + ((pw.p << SHIFT) + t - pos0);
      w = __ldg(reinterpret_cast<const uint4*>(a.k_new + src * a.k_row + head * D + 8 * cc));
      v = __ldg(reinterpret_cast<const uint4*>(a.v_new + src * a.v_row + head * D + 8 * cc));
      if (a.rope_dim > 0) cs = a.rope + static_cast<long long>((pw.p << SHIFT) + t) * a.rope_dim;
    }
    rotate8<CH>(w, kf, Angles(cs, a.rope_dim, a.interleaved, cc), a.rope_dim, a.interleaved, cc);
    bf16x8_to_f32(v, vf);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= isnan(kf[i]) || isnan(vf[i]);
    const unsigned int row_lanes = ((1u << CH) - 1u) << (lane & ~(CH - 1));
    nan_row = (__ballot_sync(0xffffffffu, bad) & row_lanes) != 0u;
  };
  const int turns = (hi - lo + kRows - 1) / kRows;
  float amax_k = 0.f, amax_v = 0.f;
#pragma unroll 2
  for (int i = 0; i < turns; ++i) {
    load(lo + i * kRows + row);
    if (nan_row) continue;
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      amax_k = fmaxf(amax_k, fabsf(kf[z]));
      amax_v = fmaxf(amax_v, fabsf(vf[z]));
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    amax_k = fmaxf(amax_k, __shfl_xor_sync(0xffffffffu, amax_k, off));
    amax_v = fmaxf(amax_v, __shfl_xor_sync(0xffffffffu, amax_v, off));
  }
  if (lane == 0) {
    red[0][warp] = amax_k;
    red[1][warp] = amax_v;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    amax_k = fmaxf(amax_k, red[0][w]);
    amax_v = fmaxf(amax_v, red[1][w]);
  }
  int ek = amax_exp(amax_k), ev = amax_exp(amax_v);
  if (lo > 0) {
    ek = max(ek, ek_old);
    ev = max(ev, ev_old);
    if (ek > ek_old) rescale_rows<D, NT>(kp, lo, exp2i(ek_old - ek));
    if (ev > ev_old) rescale_rows<D, NT>(vp, lo, exp2i(ev_old - ev));
  }
  if (tid == 0) {
    a.k_scale[sc] = exp2i(ek);
    a.v_scale[sc] = exp2i(ev);
  }
  const float mk = exp2i(-ek), mv = exp2i(-ev);
  float low[8], high[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low[i] = INFINITY;
    high[i] = -INFINITY;
  }
  for (int i = 0; i < turns; ++i) {
    const int t = lo + i * kRows + row;
    if (turns > 1) load(t);              // else its only token is still here
    if (t >= hi) continue;               // whole rows of lanes; no shuffle below
    uint2 ck, cv;
    if (nan_row) {
      ck = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      cv = make_uint2(0u, 0u);
    } else {
      ck = encode8(kf, mk);
      cv = encode8(vf, mv);
      const float4 x0 = e4m3x4_to_f32x4(ck.x), x1 = e4m3x4_to_f32x4(ck.y);
      const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        low[z] = fminf(low[z], x[z]);
        high[z] = fmaxf(high[z], x[z]);
      }
    }
    if (!dcheck(inside(t * D + 8 * cc, 8, PAGE * D), a.status, 604)) continue;
    *reinterpret_cast<uint2*>(kp + t * D + 8 * cc) = ck;
    *reinterpret_cast<uint2*>(vp + t * D + 8 * cc) = cv;
  }
  if (a.bounds != nullptr) store_bounds<D, NT>(a.bounds + sc * 2 * D, bnd, low, high, lo > 0, ek_old - ek);
}

template <int D, int SHIFT>
cudaError_t launch_t(const CacheAppendArgs& a, cudaStream_t stream) {
  const long long units = (a.s.T >> SHIFT) + 2ll * a.s.B;
  const long long items = a.q != nullptr ? static_cast<long long>(a.s.T) * ((a.Hq + kQHeads - 1) / kQHeads) : 0;
  const int per = kThreads / (D / 8);
  const long long blocks = units * a.Hkv + (items + per - 1) / per + 1;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  append_kernel<D, SHIFT><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, static_cast<int>(units));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(int page, int d, const CacheAppendArgs& a, cudaStream_t stream) {
  if (d == 64)
    return page == 32 ? launch_t<64, 5>(a, stream)
                      : (page == 64 ? launch_t<64, 6>(a, stream) : launch_t<64, 7>(a, stream));
  return page == 32 ? launch_t<128, 5>(a, stream)
                    : (page == 64 ? launch_t<128, 6>(a, stream) : launch_t<128, 7>(a, stream));
}

}  // namespace fattn
