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
// Bound: the bytes of q, k, v in and q, codes out.  One CTA of 256 threads
// takes one page of one head, K and V together, holds its up to 128 tokens in
// registers between the maximum and the quantisation, and reads each input
// once; further CTAs rotate q, one token each.
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kAppThreads = 256;

__device__ __forceinline__ void bf16x8_to_f32(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Rotates the 8 columns [8 cc, 8 cc + 8) of a row that CH = D / 8 neighbouring
// lanes hold; every lane of the warp takes part.  cs: the row's cosines and
// sines (h of each), or nullptr where there is no row.
template <int CH>
__device__ __forceinline__ void rotate8(const uint4& w, float (&f)[8], const float* cs, int rope_dim,
                                        int interleaved, int cc) {
  bf16x8_to_f32(w, f);
  if (rope_dim == 0) return;   // the same for the whole launch
  const int h = rope_dim >> 1;
  const int dim = 8 * cc;
  if (interleaved) {
    if (cs == nullptr || dim >= rope_dim) return;
    const float4 c = *reinterpret_cast<const float4*>(cs + (dim >> 1));
    const float4 s = *reinterpret_cast<const float4*>(cs + h + (dim >> 1));
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = f[2 * i], b = f[2 * i + 1];
      f[2 * i] = __fsub_rn(__fmul_rn(a, cv[i]), __fmul_rn(b, sv[i]));
      f[2 * i + 1] = __fadd_rn(__fmul_rn(b, cv[i]), __fmul_rn(a, sv[i]));
    }
    return;
  }
  // halves: column i pairs with column i + h, h / 8 chunks away
  const bool in = dim < rope_dim, low = dim < h;
  const int pc = in ? (low ? cc + (h >> 3) : cc - (h >> 3)) : cc;
  const int src = ((threadIdx.x & 31) & ~(CH - 1)) | pc;
  uint4 p;
  p.x = __shfl_sync(0xffffffffu, w.x, src);
  p.y = __shfl_sync(0xffffffffu, w.y, src);
  p.z = __shfl_sync(0xffffffffu, w.z, src);
  p.w = __shfl_sync(0xffffffffu, w.w, src);
  if (cs == nullptr || !in) return;
  float g[8];
  bf16x8_to_f32(p, g);
  const int at = low ? dim : dim - h;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 c = *reinterpret_cast<const float4*>(cs + at + 4 * q);
    const float4 s = *reinterpret_cast<const float4*>(cs + h + at + 4 * q);
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = __fmul_rn(f[4 * q + i], cv[i]), y = __fmul_rn(g[4 * q + i], sv[i]);
      f[4 * q + i] = low ? __fsub_rn(x, y) : __fadd_rn(x, y);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return pack_bf16x2(a, b); }

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
template <int D>
__device__ __forceinline__ void rescale_rows(uint8_t* base, int rows, float mul) {
  uint4* p = reinterpret_cast<uint4*>(base);
  for (int i = threadIdx.x; i < rows * (D / 16); i += kAppThreads) {
    uint4 w = p[i];
    w.x = rescale4(w.x, mul);
    w.y = rescale4(w.y, mul);
    w.z = rescale4(w.z, mul);
    w.w = rescale4(w.w, mul);
    p[i] = w;
  }
}

template <int D>
__device__ __forceinline__ void rotate_q_row(const CacheAppendArgs& a, int row) {
  constexpr int CH = D / 8;
  const int b = find_last_warp(a.s.B, row, [&](int i) { return __ldg(a.s.q_start + i); });
  const int r0 = __ldg(a.s.q_start + b), r1 = __ldg(a.s.q_start + b + 1);
  const int len = __ldg(a.s.kv_len + b);
  if (row < r0 || row >= r1) return;   // behind the last sequence
  const int pos = len - (r1 - r0) + (row - r0);
  if (pos < 0 || (a.rope_dim > 0 && pos >= a.rope_len)) {
    if (threadIdx.x == 0) record_bad_index(a.status, kSitePosition);
    return;
  }
  const float* cs = a.rope_dim > 0 ? a.rope + static_cast<long long>(pos) * a.rope_dim : nullptr;
  const int total = a.Hq * CH;
  for (int base = 0; base < total; base += kAppThreads) {
    const int ci = base + static_cast<int>(threadIdx.x);
    const bool on = ci < total;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (on) w = *reinterpret_cast<const uint4*>(a.q + row * a.q_row + 8ll * ci);
    float f[8];
    rotate8<CH>(w, f, on ? cs : nullptr, a.rope_dim, a.interleaved, ci % CH);
    if (on)
      *reinterpret_cast<uint4*>(a.q_out + (static_cast<long long>(row) * total + ci) * 8) =
          make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                     pack_bf16(f[6], f[7]));
  }
}

// Work units of the new tokens' pages: sequence b's are numbered from
// q_start[b] / PAGE + 2 b.  n tokens touch at most n / PAGE + 2 pages, so the
// ranges hold them; units past a sequence's last page do nothing.
template <int D, int PAGE>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const CacheAppendArgs a, int units) {
  constexpr int CH = D / 8;                            // 16-byte chunks of a bf16 row
  constexpr int S = PAGE * CH / kAppThreads;           // chunks of a page per thread
  constexpr int kShift = PAGE == 32 ? 5 : (PAGE == 64 ? 6 : 7);
  static_assert(PAGE * CH % kAppThreads == 0 && kAppThreads % CH == 0, "chunks per thread");
  __shared__ float red[2][kAppThreads / 32];
  __shared__ float bnd[2][kAppThreads / 32][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const long long kv_blocks = static_cast<long long>(units) * a.Hkv;
  if (blockIdx.x >= kv_blocks) {
    rotate_q_row<D>(a, static_cast<int>(blockIdx.x - kv_blocks));
    return;
  }
  const int u = blockIdx.x / a.Hkv, head = blockIdx.x - u * a.Hkv;
  auto first_unit = [&](int i) { return __ldg(a.s.q_start + i) / PAGE + 2 * i; };
  const int b = find_last_warp(a.s.B, u, first_unit);
  const SeqInfo q = seq_info(a.s, b, kShift);
  if (!q.ok) {
    if (tid == 0) record_bad_index(a.status, kSiteSeqStart);
    return;
  }
  const int nth = u - first_unit(b);
  if (nth < 0 || q.n == 0) return;
  const int pos0 = q.len - q.n;
  if (pos0 < 0 || (a.rope_dim > 0 && q.len > a.rope_len)) {
    if (tid == 0) record_bad_index(a.status, kSitePosition);
    return;
  }
  const int p = pos0 / PAGE + nth;                     // the sequence's page
  if (p >= (q.len + PAGE - 1) / PAGE) return;
  const int lo = max(pos0 - p * PAGE, 0), hi = min(q.len - p * PAGE, PAGE);   // new slots [lo, hi)
  const int pid = __ldg(a.s.table + static_cast<long long>(b) * a.s.max_pages + p);
  if (pid < 0 || pid >= a.pages) {
    if (tid == 0) record_bad_index(a.status, kSitePage);
    return;
  }
  const long long sc = static_cast<long long>(pid) * a.Hkv + head;
  const int ek_old = scale_exp(a.k_scale[sc]), ev_old = scale_exp(a.v_scale[sc]);

  // ---- the new tokens, rotated
  const int cc = tid % CH;
  float kf[S][8];
  uint4 vw[S];
  unsigned int nan_rows = 0u;                          // bit s: a token with a NaN
  float amax_k = 0.f, amax_v = 0.f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int t = (tid + s * kAppThreads) / CH;
    const bool on = t >= lo && t < hi;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    vw[s] = w;
    const float* cs = nullptr;
    if (on) {
      const long long row = q.r0 + (p * PAGE + t - pos0);
      w = *reinterpret_cast<const uint4*>(a.k_new + row * a.k_row + head * D + 8 * cc);
      vw[s] = *reinterpret_cast<const uint4*>(a.v_new + row * a.v_row + head * D + 8 * cc);
      if (a.rope_dim > 0) cs = a.rope + static_cast<long long>(p * PAGE + t) * a.rope_dim;
    }
    rotate8<CH>(w, kf[s], cs, a.rope_dim, a.interleaved, cc);
    float vf[8];
    bf16x8_to_f32(vw[s], vf);
    bool bad = false;
    float mk = 0.f, mv = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bad |= isnan(kf[s][i]) || isnan(vf[i]);
      mk = fmaxf(mk, fabsf(kf[s][i]));
      mv = fmaxf(mv, fabsf(vf[i]));
    }
    const unsigned int row_lanes = ((1u << CH) - 1u) << (lane & ~(CH - 1));
    if (__ballot_sync(0xffffffffu, bad) & row_lanes) {
      nan_rows |= 1u << s;
    } else {
      amax_k = fmaxf(amax_k, mk);
      amax_v = fmaxf(amax_v, mv);
    }
  }

  // ---- the page's scales
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
  amax_k = red[0][0];
  amax_v = red[1][0];
#pragma unroll
  for (int w = 1; w < kAppThreads / 32; ++w) {
    amax_k = fmaxf(amax_k, red[0][w]);
    amax_v = fmaxf(amax_v, red[1][w]);
  }
  int ek = amax_exp(amax_k), ev = amax_exp(amax_v);
  uint8_t* kp = a.k + pid * a.page_stride + static_cast<long long>(head) * PAGE * D;
  uint8_t* vp = a.v + pid * a.page_stride + static_cast<long long>(head) * PAGE * D;
  if (lo > 0) {
    ek = max(ek, ek_old);
    ev = max(ev, ev_old);
    if (ek > ek_old) rescale_rows<D>(kp, lo, exp2i(ek_old - ek));
    if (ev > ev_old) rescale_rows<D>(vp, lo, exp2i(ev_old - ev));
  }
  if (tid == 0) {
    a.k_scale[sc] = exp2i(ek);
    a.v_scale[sc] = exp2i(ev);
  }

  // ---- codes, and the extremes of the keys' codes per column
  const float mk = exp2i(-ek), mv = exp2i(-ev);
  float low[8], high[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low[i] = INFINITY;
    high[i] = -INFINITY;
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int t = (tid + s * kAppThreads) / CH;
    if (t < lo || t >= hi) continue;
    uint2 ck, cv;
    if (nan_rows >> s & 1u) {
      // NaN in a key or a value: the token's key is NaN and its value zero,
      // so that every row that attends to it is NaN and no other row is.
      ck = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      cv = make_uint2(0u, 0u);
    } else {
      ck = encode8(kf[s], mk);
      float vf[8];
      bf16x8_to_f32(vw[s], vf);
      cv = encode8(vf, mv);
      if (a.bounds != nullptr) {
        const float4 x0 = e4m3x4_to_f32x4(ck.x), x1 = e4m3x4_to_f32x4(ck.y);
        const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          low[i] = fminf(low[i], x[i]);
          high[i] = fmaxf(high[i], x[i]);
        }
      }
    }
    *reinterpret_cast<uint2*>(kp + t * D + 8 * cc) = ck;
    *reinterpret_cast<uint2*>(vp + t * D + 8 * cc) = cv;
  }
  if (a.bounds == nullptr) return;
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
  if (tid < 2 * D) {
    const int side = tid / D, col = tid % D;
    float x = bnd[side][0][col];
#pragma unroll
    for (int w = 1; w < kAppThreads / 32; ++w)
      x = side ? fmaxf(x, bnd[side][w][col]) : fminf(x, bnd[side][w][col]);
    // rounded outwards: a page's bounds stay bounds
    if (isfinite(x)) x = side ? ceilf(bound_units(x)) : floorf(bound_units(x));
    int8_t* out = a.bounds + (sc * 2 + side) * D + col;
    if (lo > 0) {
      const float old = __fmul_rn(static_cast<float>(*out), exp2i(ek_old - ek));
      x = side ? fmaxf(x, ceilf(old)) : fminf(x, floorf(old));
    }
    if (!isfinite(x)) x = 0.f;   // a fresh page of NaN tokens alone
    *out = static_cast<int8_t>(x);
  }
}

template <int D, int PAGE>
cudaError_t launch_t(const CacheAppendArgs& a, cudaStream_t stream) {
  const long long units = a.s.T / PAGE + 2ll * a.s.B;
  const long long blocks = units * a.Hkv + (a.q != nullptr ? a.s.T : 0);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  append_kernel<D, PAGE><<<static_cast<unsigned>(blocks), kAppThreads, 0, stream>>>(
      a, static_cast<int>(units));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(int page, int d, const CacheAppendArgs& a, cudaStream_t stream) {
  if (d == 64)
    return page == 32 ? launch_t<64, 32>(a, stream)
                      : (page == 64 ? launch_t<64, 64>(a, stream) : launch_t<64, 128>(a, stream));
  return page == 32 ? launch_t<128, 32>(a, stream)
                    : (page == 64 ? launch_t<128, 64>(a, stream) : launch_t<128, 128>(a, stream));
}

}  // namespace fattn
