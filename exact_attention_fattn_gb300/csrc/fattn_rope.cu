// Rotary positions: the pairs (a, b) of a row's first rope_dim columns become
// (a cos - b sin, b cos + a sin), angles from an fp32 table by the row's
// position; transposed (sin negated) for gradients, since dx = R^T dy.  fp32,
// products and sums rounded one by one, so that the result does not depend on
// what a compiler contracts, then one rounding to bf16.
//
// Bound: the bytes of x and y.  A thread has 8 pairs (two 16-byte loads) of up to
// four heads of one row, so that their cosines and sines are loaded once and the
// heads' loads go out together; neighbouring threads have a row's neighbouring
// pairs, then rows or heads, whichever lie closer.  Measured, [2, 32, 4096, 128] (136 MB):
// 21.7 us, 0.93 of the measured copy rate (two heads a thread 22.0, eight 24.8); a
// few rows 2.8 us.
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/fattn.h"
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr int kHeads = 4;      // heads of a thread, at most
constexpr int kThreads = 256;

struct RopeArgs {
  const uint16_t* x;
  uint16_t* y;
  long long xb, xh, xn, yb, yh, yn;   // strides, elements
  const float* rope;
  int rope_len, rope_dim, interleaved, transposed;
  const int* positions;               // or nullptr: the row's index
  long long pos_stride;
  int B, H, N, d;
  int items;                          // 16 columns each, of a row; those to rotate first
  int per, groups;                    // heads of a thread, threads for a row's heads
  int heads_first;                    // neighbouring threads: heads before rows
  int small;                          // threads are numbered in 32 bits
  DeviceStatus* status;
};

__device__ __forceinline__ void rotate_pair(uint32_t& wa, uint32_t& wb, float c0, float s0, float c1, float s1) {
  const float a0 = __uint_as_float(wa << 16), a1 = __uint_as_float(wa & 0xffff0000u);
  const float b0 = __uint_as_float(wb << 16), b1 = __uint_as_float(wb & 0xffff0000u);
  wa = pack_bf16x2(__fsub_rn(__fmul_rn(a0, c0), __fmul_rn(b0, s0)),
                   __fsub_rn(__fmul_rn(a1, c1), __fmul_rn(b1, s1)));
  wb = pack_bf16x2(__fadd_rn(__fmul_rn(b0, c0), __fmul_rn(a0, s0)),
                   __fadd_rn(__fmul_rn(b1, c1), __fmul_rn(a1, s1)));
}

// Neighbouring pairs: a word is (a, b).
__device__ __forceinline__ void rotate_word(uint32_t& w, float c, float s) {
  const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xffff0000u);
  w = pack_bf16x2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  const long long at = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int inner = a.heads_first ? a.groups : a.N, outer = a.heads_first ? a.N : a.groups;
  int item, i, o, b;
  if (a.small) {                          // 64-bit divisions cost several times as much
    unsigned int t = static_cast<unsigned int>(at);
    item = t % a.items;
    t /= a.items;
    i = t % inner;
    t /= inner;
    o = t % outer;
    b = t / outer;
  } else {
    long long t = at / a.items;
    item = static_cast<int>(at % a.items);
    i = static_cast<int>(t % inner);
    t /= inner;
    o = static_cast<int>(t % outer);
    b = static_cast<int>(t / outer);
  }
  if (b >= a.B) return;
  const int n = a.heads_first ? o : i, g = a.heads_first ? i : o;
  const int pos = a.positions != nullptr ? __ldg(a.positions + b * a.pos_stride + n) : n;
  if (pos < 0 || pos >= a.rope_len) {
    record_bad_index(a.status, kSitePosition);
    return;
  }
  const bool turn = item < a.rope_dim / 16;
  const int half = a.rope_dim / 2;
  const int c0 = turn && !a.interleaved ? 8 * item : 16 * item;
  const int c1 = turn && !a.interleaved ? half + 8 * item : 16 * item + 8;
  const int h0 = g * a.per, h1 = min(a.H, h0 + a.per);
  const uint16_t* x = a.x + b * a.xb + n * a.xn + h0 * a.xh;
  uint16_t* y = a.y + b * a.yb + n * a.yn + h0 * a.yh;
  if (!dcheck(inside(c0, 8, a.d) && inside(c1, 8, a.d) && h0 < a.H, a.status, 661)) return;
  uint4 u[kHeads], v[kHeads];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k >= h1) break;
    u[k] = *reinterpret_cast<const uint4*>(x + k * a.xh + c0);
    v[k] = *reinterpret_cast<const uint4*>(x + k * a.xh + c1);
  }
  if (turn) {
    const float4* cs = reinterpret_cast<const float4*>(a.rope + static_cast<long long>(pos) * a.rope_dim + 8 * item);
    const float4* sn = reinterpret_cast<const float4*>(a.rope + static_cast<long long>(pos) * a.rope_dim + half + 8 * item);
    const float4 p = __ldg(cs), q = __ldg(cs + 1);
    float4 r = __ldg(sn), s = __ldg(sn + 1);
    if (a.transposed) {
      r = make_float4(-r.x, -r.y, -r.z, -r.w);
      s = make_float4(-s.x, -s.y, -s.z, -s.w);
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h0 + k >= h1) break;
      if (a.interleaved) {
        rotate_word(u[k].x, p.x, r.x);
        rotate_word(u[k].y, p.y, r.y);
        rotate_word(u[k].z, p.z, r.z);
        rotate_word(u[k].w, p.w, r.w);
        rotate_word(v[k].x, q.x, s.x);
        rotate_word(v[k].y, q.y, s.y);
        rotate_word(v[k].z, q.z, s.z);
        rotate_word(v[k].w, q.w, s.w);
      } else {
        rotate_pair(u[k].x, v[k].x, p.x, r.x, p.y, r.y);
        rotate_pair(u[k].y, v[k].y, p.z, r.z, p.w, r.w);
        rotate_pair(u[k].z, v[k].z, q.x, s.x, q.y, s.y);
        rotate_pair(u[k].w, v[k].w, q.z, s.z, q.w, s.w);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    if (h0 + k >= h1) break;
    *reinterpret_cast<uint4*>(y + k * a.yh + c0) = u[k];
    *reinterpret_cast<uint4*>(y + k * a.yh + c1) = v[k];
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides of a [B, H, N, d] view whose rows are whole: multiples of 8, and below
// 2^40 so that no offset overflows.  Rows that are written do not overlap.
bool strides_ok(const long long* s, int B, int H, int N, int d, bool written) {
  const int n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (s[i] % 8 != 0 || s[i] < 0 || s[i] >= (1ll << 40)) return false;
    if (written && n[i] > 1 && s[i] < d) return false;
  }
  if (!written) return true;
  // each extent lies within the next larger stride (a dense or a sliced layout)
  int o[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[o[j]] > s[o[j + 1]]) {
        const int x = o[j];
        o[j] = o[j + 1];
        o[j + 1] = x;
      }
  long long reach = d;
  for (int i = 0; i < 3; ++i) {
    if (n[o[i]] == 1) continue;
    if (s[o[i]] < reach) return false;
    reach += s[o[i]] * (n[o[i]] - 1);
  }
  return true;
}

}  // namespace

}  // namespace fattn

using namespace fattn;

extern "C" int fattn_rope(const void* x, long long x_b, long long x_h, long long x_n, void* y, long long y_b,
                          long long y_h, long long y_n, const float* rope, int rope_len, int rope_dim, int interleaved,
                          int transposed, const int* positions, long long positions_b, int B, int H, int N, int d,
                          fattn_stream_t stream) {
  struct Range {
    Range() { nvtxRangePushA("fattn_rope"); }
    ~Range() { nvtxRangePop(); }
  } const range;
  if (d <= 0 || d > 1024 || d % 16 != 0) return FATTN_ERR_UNSUPPORTED;
  if (B <= 0 || H <= 0 || N <= 0 || !x || !y || !rope) return FATTN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(rope, 16) || !aligned(positions, 4)) return FATTN_ERR_INVALID_ARG;
  if (rope_len <= 0 || rope_dim <= 0 || rope_dim > d || rope_dim % 16 != 0) return FATTN_ERR_INVALID_ARG;
  if (positions_b < 0 || positions_b >= (1ll << 40)) return FATTN_ERR_INVALID_ARG;
  const long long x_strides[3] = {x_b, x_h, x_n}, y_strides[3] = {y_b, y_h, y_n};
  if (!strides_ok(x_strides, B, H, N, d, false) || !strides_ok(y_strides, B, H, N, d, true))
    return FATTN_ERR_INVALID_ARG;
  const bool same = x == y;
  for (int i = 0; i < 3; ++i) {
    const int n = i == 0 ? B : (i == 1 ? H : N);
    if (same && n > 1 && x_strides[i] != y_strides[i]) return FATTN_ERR_INVALID_ARG;
  }
  RopeArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.y = static_cast<uint16_t*>(y);
  a.xb = x_b, a.xh = x_h, a.xn = x_n;
  a.yb = y_b, a.yh = y_h, a.yn = y_n;
  a.rope = rope;
  a.rope_len = rope_len;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved != 0;
  a.transposed = transposed != 0;
  a.positions = positions;
  a.pos_stride = positions_b;
  a.B = B, a.H = H, a.N = N, a.d = d;
  a.items = (same ? rope_dim : d) / 16;
  // Four heads a thread where that leaves work for all SMs, one where it does not.
  const long long rows = static_cast<long long>(B) * N;
  a.per = 1;
  while (a.per < kHeads && a.per < H && rows * a.items * ((H + 2 * a.per - 1) / (2 * a.per)) >= kSms * 2048ll) a.per *= 2;
  a.groups = (H + a.per - 1) / a.per;
  a.heads_first = a.xh < a.xn;
  const long long lanes = rows * a.items * a.groups, blocks = (lanes + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return FATTN_ERR_TOO_LARGE;
  a.small = blocks * kThreads < (1ll << 32);
  long long budget = 0;
  const int rc = call_setup(&a.status, &budget);
  if (rc != FATTN_OK) return rc;
  rope_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FATTN_OK : FATTN_ERR_CUDA;
}
