// Second kernel of the attention over the paged 8-bit cache: units whose keys
// several CTAs shared are put together from the parts they left in the
// workspace (unnormalised rows of O in fp32, reference maximum and sum).
#include "fattn_cache.cuh"

namespace fattn {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;

// Joins the partial results of the units that several CTAs share, in the
// order of their keys: block (c, y) takes two rows of the unit that goes on
// after CTA c.  Four groups of D / 4 threads a row walk the parts.
template <int D, int ROWS>
__global__ void __launch_bounds__(2 * D) join_kernel(const CacheAttnArgs a) {
  constexpr int kF4 = D / 4, kGroups = 4, kRowsPerBlock = 2;
  static_assert(kF4 * kGroups * kRowsPerBlock == 2 * D, "threads");
  __shared__ float4 part[kGroups][kRowsPerBlock][kF4];
  __shared__ float2 pml[kGroups][kRowsPerBlock];
  const int cta = blockIdx.x, G = a.grid;
  const int4 rec = a.rec[2 * cta];
  if (rec.y == 0) return;                            // nothing shared from here
  const int4 more = a.rec[2 * cta + 1];
  const long long W = (static_cast<long long>(more.z) << 32) | static_cast<unsigned int>(more.y);
  const int q4 = threadIdx.x % kF4, local = threadIdx.x / kF4 % kRowsPerBlock;
  const int group = threadIdx.x / (kF4 * kRowsPerBlock);
  const int row = blockIdx.y * kRowsPerBlock + local;
  const long long rr = static_cast<long long>(rec.z) * ROWS + row;
  const bool on = rr < static_cast<long long>(rec.y) * a.group;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = cta + group; on && p <= more.x; p += kGroups) {
    if (cta_first(W, G, p) == cta_first(W, G, p + 1)) continue;   // a CTA without work
    const long long slot = 2ll * p + (p == cta ? 1 : 0);
    const float2 x = a.part_ml[slot * ROWS + row];
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (slot * ROWS + row) * D + 4 * q4);
    const float n = fmaxf(m, x.x);
    const float b0 = n == -INFINITY ? 1.f : ex2_approx(m - n);
    const float b1 = n == -INFINITY ? 1.f : ex2_approx(x.x - n);
    m = n;
    l = fmaf(l, b0, x.y * b1);
    acc.x = fmaf(acc.x, b0, v.x * b1);
    acc.y = fmaf(acc.y, b0, v.y * b1);
    acc.z = fmaf(acc.z, b0, v.z * b1);
    acc.w = fmaf(acc.w, b0, v.w * b1);
  }
  part[group][local][q4] = acc;
  if (q4 == 0) pml[group][local] = make_float2(m, l);
  __syncthreads();
  if (group != 0 || !on) return;
#pragma unroll
  for (int g = 1; g < kGroups; ++g) {
    const float2 x = pml[g][local];
    const float4 v = part[g][local][q4];
    const float n = fmaxf(m, x.x);
    const float b0 = n == -INFINITY ? 1.f : ex2_approx(m - n);
    const float b1 = n == -INFINITY ? 1.f : ex2_approx(x.x - n);
    m = n;
    l = fmaf(l, b0, x.y * b1);
    acc.x = fmaf(acc.x, b0, v.x * b1);
    acc.y = fmaf(acc.y, b0, v.y * b1);
    acc.z = fmaf(acc.z, b0, v.z * b1);
    acc.w = fmaf(acc.w, b0, v.w * b1);
  }
  const int token = static_cast<int>(rr / a.group);
  const long long at = (static_cast<long long>(rec.x + token) * a.Hkv + rec.w) * a.group +
                       (rr - static_cast<long long>(token) * a.group);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(a.o + at * D + 4 * q4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (q4 == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, int ROWS>
cudaError_t launch_t(const CacheAttnArgs& a, cudaStream_t stream) {
  join_kernel<D, ROWS><<<dim3(a.grid, ROWS / 2), 2 * D, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_join(int d, int rows, const CacheAttnArgs& a, cudaStream_t stream) {
  if (rows == kDecodeRows)
    return d == 64 ? launch_t<64, kDecodeRows>(a, stream) : launch_t<128, kDecodeRows>(a, stream);
  return d == 64 ? launch_t<64, kChunkRows>(a, stream) : launch_t<128, kChunkRows>(a, stream);
}

}  // namespace fattn
