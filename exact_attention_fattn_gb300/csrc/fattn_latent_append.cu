// Appending to the paged latent cache: a token's latent vector and its key part,
// rotated by its position, go to its slot, and its queries' rotated parts into
// their place behind the absorbed ones.  Rotation as in the 8-bit cache: fp32,
// every product and sum rounded, one rounding to bf16.
//
// Bound: the bytes in and out.  A warp has a token's row (a 16-byte load a lane and
// 256 columns, and one of 4 lanes for the key part's 16 columns each); further
// threads have 16 columns of two heads' query parts.  Measured, 3 prompts of 3500 to
// 4096 tokens, 64 heads, rank 512 (218 MB): 39.1 us, 0.82 of the measured copy rate
// (one head a thread 42.1, four 39.9, eight 43.7; 256 threads a block 40.4); 32
// tokens of as many sequences 2.5 us.
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 2;
constexpr int kItems = kLatentRope / 16;   // 16 columns, 8 pairs each

__device__ __forceinline__ bool finite_words(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) ok &= (u[i] & 0x7f80u) != 0x7f80u && (u[i] & 0x7f800000u) != 0x7f800000u;
  return ok;
}

// Columns 8 i .. 8 i + 7 of both halves (u, v), or 16 i .. 16 i + 15 when interleaved.
struct Turn {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* rope, int pos, int item) {
    const float4* p = reinterpret_cast<const float4*>(rope + static_cast<long long>(pos) * kLatentRope + 8 * item);
    const float4 a = __ldg(p), b = __ldg(p + 1), d = __ldg(p + 8), e = __ldg(p + 9);   // sines 32 floats on
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
    s[0] = d.x, s[1] = d.y, s[2] = d.z, s[3] = d.w, s[4] = e.x, s[5] = e.y, s[6] = e.z, s[7] = e.w;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ float first(float a, float b, float c, float s) {
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  }
  static __device__ __forceinline__ float second(float a, float b, float c, float s) {
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  }
  __device__ __forceinline__ void apply(uint4& u, uint4& v, bool interleaved) const {
    uint32_t x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = pack_bf16x2(first(lo(x[i]), hi(x[i]), c[i], s[i]), second(lo(x[i]), hi(x[i]), c[i], s[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = x[i], b = x[4 + i];
        x[i] = pack_bf16x2(first(lo(a), lo(b), c[2 * i], s[2 * i]), first(hi(a), hi(b), c[2 * i + 1], s[2 * i + 1]));
        x[4 + i] = pack_bf16x2(second(lo(a), lo(b), c[2 * i], s[2 * i]), second(hi(a), hi(b), c[2 * i + 1], s[2 * i + 1]));
      }
    }
    u = make_uint4(x[0], x[1], x[2], x[3]);
    v = make_uint4(x[4], x[5], x[6], x[7]);
  }
};

// The sequence of a token, its position, and whether the call takes it.
struct Token {
  int b, pos;
  bool ok;
};

__device__ __forceinline__ Token token_of(const LatentAppendArgs& a, int token) {
  // a guess for sequences of equal rows, else a search
  int b = static_cast<int>(static_cast<long long>(token) * a.s.B / a.s.T);
  if (token < __ldg(a.s.q_start + b) || token >= __ldg(a.s.q_start + b + 1)) {
    b = 0;
    for (int hi = a.s.B; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (__ldg(a.s.q_start + mid) <= token) b = mid; else hi = mid;
    }
  }
  const SeqInfo q = seq_info(a.s, b, a.page_shift);
  Token t{b, q.len - q.n + token - q.r0, token >= q.r0 && token < q.r0 + q.n};
  if (t.ok && (q.len < q.n || (a.rope != nullptr && q.len > a.rope_len))) {
    record_bad_index(a.status, kSitePosition);
    t.ok = false;
  }
  return t;
}

__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ LatentAppendArgs a, int key_blocks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = lane & (kItems - 1);
  const int c0 = a.interleaved ? 16 * item : 8 * item, c1 = a.interleaved ? c0 + 8 : kLatentRope / 2 + c0;
  if (static_cast<int>(blockIdx.x) == key_blocks) {
    check_seqs(a.s, threadIdx.x, kThreads, a.page_shift, a.status);
    return;
  }
  if (static_cast<int>(blockIdx.x) > key_blocks) {
    // ---- query parts
    const int groups = (a.Hq + kHeads - 1) / kHeads;
    const long long id = (static_cast<long long>(blockIdx.x - key_blocks - 1) * kThreads + threadIdx.x) / kItems;
    const int token = static_cast<int>(id / groups), h0 = static_cast<int>(id - static_cast<long long>(token) * groups) * kHeads;
    if (token >= a.s.T) return;
    const uint16_t* src = a.q_rope + token * a.qr_row + h0 * a.qr_head;
    uint4 u[kHeads], v[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const long long off = min(k, a.Hq - 1 - h0) * a.qr_head;
      // q may be the same columns, so these are no read-only data
      u[k] = *reinterpret_cast<const uint4*>(src + off + c0);
      v[k] = *reinterpret_cast<const uint4*>(src + off + c1);
    }
    const Token t = token_of(a, token);
    if (!t.ok) return;
    Turn turn;
    if (a.rope != nullptr) turn.load(a.rope, t.pos, item);
    const int width = a.rank + kLatentRope;
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h0 + k >= a.Hq) break;
      if (a.rope != nullptr) turn.apply(u[k], v[k], a.interleaved);
      if (!dcheck(inside(h0 + k, 1, a.Hq) && inside(token, 1, a.s.T), a.status, 681)) continue;
      uint16_t* dst = a.q + (static_cast<long long>(token) * a.Hq + h0 + k) * width + a.rank;
      *reinterpret_cast<uint4*>(dst + c0) = u[k];
      *reinterpret_cast<uint4*>(dst + c1) = v[k];
    }
    return;
  }
  // ---- latent and key part of a token, a warp each
  const long long id = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  if (id >= a.s.T) return;
  const int token = static_cast<int>(id);
  const uint16_t* src = a.latent + token * a.latent_row;
  uint4 w[2] = {}, u = {}, v = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (256 * i < a.rank) w[i] = __ldg(reinterpret_cast<const uint4*>(src + 256 * i + 8 * lane));
  if (lane < kItems) {
    u = __ldg(reinterpret_cast<const uint4*>(a.k_rope + token * a.k_row + c0));
    v = __ldg(reinterpret_cast<const uint4*>(a.k_rope + token * a.k_row + c1));
  }
  const Token t = token_of(a, token);
  if (!t.ok) return;                      // the warp's lanes have the same token
  const int page = __ldg(a.s.table + static_cast<long long>(t.b) * a.s.max_pages + (t.pos >> a.page_shift));
  if (page < 0 || page >= a.pages) {
    if (lane == 0) record_bad_index(a.status, kSitePage);
    return;
  }
  if (lane < kItems && a.rope != nullptr) {
    Turn turn;
    turn.load(a.rope, t.pos, item);
    turn.apply(u, v, a.interleaved);
  }
  // A latent is its token's value, too, and a masked probability of zero times an
  // infinity or a NaN is a NaN: such a token gets a NaN key part and a zero latent.
  const bool fine = finite_words(w[0]) && finite_words(w[1]) && finite_words(u) && finite_words(v);
  if (!__all_sync(0xffffffffu, fine)) {
    w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
    u = v = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
  }
  const int width = a.rank + kLatentRope, slot = t.pos & ((1 << a.page_shift) - 1);
  if (!dcheck(inside(static_cast<long long>(slot + 1) * width, 0, a.page_stride), a.status, 682)) return;
  uint16_t* dst = a.data + page * a.page_stride + slot * width;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (256 * i < a.rank) *reinterpret_cast<uint4*>(dst + 256 * i + 8 * lane) = w[i];
  if (lane < kItems) {
    *reinterpret_cast<uint4*>(dst + a.rank + c0) = u;
    *reinterpret_cast<uint4*>(dst + a.rank + c1) = v;
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, cudaStream_t stream) {
  const long long keys = (static_cast<long long>(a.s.T) + kThreads / 32 - 1) / (kThreads / 32);
  const long long items = a.q_rope != nullptr ? static_cast<long long>(a.s.T) * ((a.Hq + kHeads - 1) / kHeads) * kItems : 0;
  const long long blocks = keys + 1 + (items + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  append_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, static_cast<int>(keys));
  return cudaGetLastError();
}

}  // namespace fattn
