// Second kernel of the attention over the paged 8-bit cache: units whose keys
// several CTAs shared are put together from the parts they left in the
// workspace (unnormalised rows of O in fp32, reference maximum and sum), in
// the order of their keys.
//
// Bound: latency where a unit has many parts (one long sequence: as many as the
// few-rows kernel has CTAs, 304, or 456 for d = 64), bytes where units are large
// (256 rows, two or three parts each).  A thread has 4 columns of a row; the small
// units' parts are walked by four groups of threads side by side, the large ones'
// by one, two rows a thread whose loads go out together (32 sequences of 40 rows,
// whole call: 67.1 us with one row, 66.5 with two, 68.1 with four).
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;

struct Part {
  float m, l;
  float4 o;
};

__device__ __forceinline__ void merge(Part& a, const Part& b) {
  const float m = fmaxf(a.m, b.m), m0 = m == -INFINITY ? 0.f : m;
  const float x = ex2_approx(a.m - m0), y = ex2_approx(b.m - m0);
  a.m = m;
  a.l = fmaf(a.l, x, b.l * y);
  a.o.x = fmaf(a.o.x, x, b.o.x * y);
  a.o.y = fmaf(a.o.y, x, b.o.y * y);
  a.o.z = fmaf(a.o.z, x, b.o.z * y);
  a.o.w = fmaf(a.o.w, x, b.o.w * y);
}

// Block (c, y): rows [y kBlock, ..) of the unit that CTA c starts and others go
// on with.
template <int D, int ROWS>
struct JoinCfg {
  static constexpr int kF4 = D / 4;                            // threads per row
  static constexpr int kGroups = ROWS == kDecodeRows ? 4 : 1;
  static constexpr int kRows = ROWS == kDecodeRows ? 4 : 8;    // rows at a time
  static constexpr int kPer = ROWS == kDecodeRows ? 1 : 2;     // rows per thread
  static constexpr int kBlock = kRows * kPer;
  static constexpr int kThreads = kF4 * kGroups * kRows;
};

template <int D, int ROWS>
__global__ void __launch_bounds__(JoinCfg<D, ROWS>::kThreads) join_kernel(const CacheAttnArgs a) {
  using J = JoinCfg<D, ROWS>;
  [[maybe_unused]] constexpr long long kPartRows = part_rows(D, ROWS);
  __shared__ Part side[J::kGroups][J::kRows][J::kF4];
  const int cta = blockIdx.x, G = a.grid;
  wait_for_parent();
  const int4 rec = a.rec[2 * cta];
  const int rows = rec.y * a.group - rec.z * ROWS;   // of the unit, from its first
  if (rec.y == 0 || static_cast<int>(blockIdx.y) * J::kBlock >= rows) return;
  const int4 more = a.rec[2 * cta + 1];
  const long long W = (static_cast<long long>(more.z) << 32) | static_cast<unsigned int>(more.y);
  const int q4 = threadIdx.x % J::kF4, local = threadIdx.x / J::kF4 % J::kRows;
  const int group = threadIdx.x / (J::kF4 * J::kRows);
  const int row0 = blockIdx.y * J::kBlock + local, end = min(rows, ROWS);
  Part p[J::kPer];
#pragma unroll
  for (int k = 0; k < J::kPer; ++k) p[k] = Part{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int c = cta + group; c <= more.x; c += J::kGroups) {
    if (cta_first(W, G, c) == cta_first(W, G, c + 1)) continue;   // a CTA without work
    const long long at = (2ll * c + (c == cta ? 1 : 0)) * ROWS;
    Part x[J::kPer] = {};
#pragma unroll
    for (int k = 0; k < J::kPer; ++k) {
      const int row = min(row0 + k * J::kRows, end - 1);          // a row that is there, to load
      if (!dcheck(row >= 0 && inside(at + row, 1, kPartRows), a.status, 621)) continue;
      const float2 ml = a.part_ml[at + row];
      x[k] = Part{ml.x, ml.y, reinterpret_cast<const float4*>(a.part_o + (at + row) * D)[q4]};
    }
#pragma unroll
    for (int k = 0; k < J::kPer; ++k) merge(p[k], x[k]);
  }
  if constexpr (J::kGroups > 1) {
    static_assert(J::kPer == 1, "one row a thread");
    side[group][local][q4] = p[0];
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 1; g < J::kGroups; ++g) merge(p[0], side[g][local][q4]);
  }
#pragma unroll
  for (int k = 0; k < J::kPer; ++k) {
    const int row = row0 + k * J::kRows;
    if (row >= end) continue;
    const int rr = rec.z * ROWS + row, token = rr / a.group;
    const long long out = (static_cast<long long>(rec.x + token) * a.Hkv + rec.w) * a.group +
                          (rr - token * a.group);
    if (!dcheck(inside(out, 1, static_cast<long long>(a.s.T) * a.Hkv * a.group), a.status, 622)) continue;
    const float inv = p[k].l == 0.f ? 0.f : 1.f / p[k].l;
    *reinterpret_cast<uint2*>(a.o + out * D + 4 * q4) = make_uint2(
        pack_bf16x2(p[k].o.x * inv, p[k].o.y * inv), pack_bf16x2(p[k].o.z * inv, p[k].o.w * inv));
    if (q4 == 0) a.lse[out] = p[k].l == 0.f ? -INFINITY : (p[k].m + log2f(p[k].l)) * kLn2;
  }
}

template <int D, int ROWS>
cudaError_t launch_t(const CacheAttnArgs& a, cudaStream_t stream) {
  using J = JoinCfg<D, ROWS>;
  static_assert(J::kThreads <= 1024, "block size");
  return launch_child(join_kernel<D, ROWS>, dim3(a.grid, ROWS / J::kBlock), J::kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_cache_join(int d, int rows, const CacheAttnArgs& a, cudaStream_t stream) {
  if (rows == kDecodeRows)
    return d == 64 ? launch_t<64, kDecodeRows>(a, stream) : launch_t<128, kDecodeRows>(a, stream);
  return d == 64 ? launch_t<64, kChunkRows>(a, stream) : launch_t<128, kChunkRows>(a, stream);
}

}  // namespace fattn
