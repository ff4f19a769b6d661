// Host-side declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fattn_smem_limit.h"

namespace fattn {

struct DeviceStatus;

// Everything a forward launch needs besides the tensor maps.
struct FwdArgs {
  uint16_t* o;                // bf16 [BH, N, d]
  float* lse;                 // [BH, N]
  DeviceStatus* status;
  long long wait_budget;      // cycles
  int N;
  int BH;
  int sec_heads;              // heads per scheduling section (set by the launcher)
  float scale_log2;           // scale * log2(e)
  float tau_log2;             // rescale threshold (log2 units)
  // FP8 only (nullptr otherwise): block scales [BH, ceil(N/128)] of Q, K, V
  const float* sq;
  const float* sk;
  const float* sv;
};

// Launch the forward kernel for head dim d (64/128).  Tensor maps are 3-D
// {d, N, B*H} views of q, k, v with 128-row boxes and a 128-byte swizzle.
cudaError_t launch_fwd(int d, bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                       const CUtensorMap& tv, const FwdArgs& a, cudaStream_t stream);

// FP8 forward (d = 128): tq, tk are 3-D uint8 views {d, N, B*H} of the e4m3
// codes with 128-byte x 128-row boxes; tv a 3-D uint8 view {Np, d, B*H} of the
// transposed V codes with the same box.
cudaError_t launch_fwd_fp8(bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const FwdArgs& a, cudaStream_t stream);

// Block quantization to e4m3: one scale per 128 rows of a head (amax / 448),
// codes [BH, N, d] or, transposed, [BH, d, Np] with zero codes past N.
cudaError_t launch_fp8_quantize(const void* x, void* codes, float* scales, int BH, int N, int d,
                                bool transpose, cudaStream_t stream);

// The same after the randomized Hadamard rotation diag(signs) H / sqrt(d) of
// every row (d = 128; not transposed).
cudaError_t launch_fp8_quantize_rotated(const void* x, const float* signs, void* codes,
                                        float* scales, int BH, int N, int d,
                                        cudaStream_t stream);

// Capacity of the backward's tail tables (kernel parameters, ~2.6 KB).
constexpr int kBwdTailMaxCtas = 256;
constexpr int kBwdTailCap = 1024;

struct BwdArgs {
  const float* L2;            // [BH, Np]: -lse * log2(e), -inf past N (Np = N rounded up to 128)
  const float* D;             // [BH, Np]: rowsum(dO o O), 0 past N
  float* dq_accum;            // [BH, N, d] fp32
  uint32_t* dq_order;         // [BH, n_tiles] contribution counters, or nullptr (any order)
  uint16_t* dk;               // bf16 [BH, N, d]
  uint16_t* dv;               // bf16 [BH, N, d]
  DeviceStatus* status;
  long long wait_budget;
  int N;
  int BH;
  int sec_heads;              // heads per scheduling section (set by the launcher)
  int paired;                 // causal K/V tiles p and n - 1 - p paired (set by the launcher)
  float scale;
  float scale_log2;
  // Paired causal schedule only (set by the launcher, see bwd_item): the
  // last tail_heads heads are dealt K/V tile by K/V tile from these tables.
  int tail_heads;
  uint16_t tail_off[kBwdTailMaxCtas + 1];  // CTA c: entries [tail_off[c], tail_off[c + 1])
  uint16_t tail_item[kBwdTailCap];         // r * n_tiles + j: K/V tile j of head BH - tail_heads + r
};

// D (and, when L2 != nullptr, L2 = -lse * log2 e) in a [BH, pitch] layout with
// padding rows N..pitch-1; zeroes dq_accum [BH, N, d] and, when given, the
// [BH, pitch / 128] dQ contribution counters.
cudaError_t launch_bwd_preprocess(const void* o, const void* dO, const float* lse, float* D,
                                  float* L2, float* dq_accum, uint32_t* counters, int BH, int N,
                                  int pitch, int d, cudaStream_t stream);

// tacc: 3-D fp32 view {d, N, B*H} of the dQ accumulator, 32 x 32 boxes,
// 128-byte swizzle (the target of the dQ reduce-adds).
cudaError_t launch_bwd_main(int d, bool causal, const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, const CUtensorMap& tdo,
                            const CUtensorMap& tacc, const BwdArgs& a, cudaStream_t stream);

// CTA-pair version of the main backward kernel (d = 128, any-order dQ; see
// fattn_bwd2.cu).  tq64 / tdo64: views of q and dO with 64-row boxes.
cudaError_t launch_bwd2_main(bool causal, const CUtensorMap& tq, const CUtensorMap& tq64,
                             const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                             const CUtensorMap& tdo64, const CUtensorMap& tacc, const BwdArgs& a,
                             cudaStream_t stream);

cudaError_t launch_dq_convert(const float* dq_accum, void* dq, long long elems, float scale,
                              cudaStream_t stream);

// ------------------------------------------------------------------ paged 8-bit cache

// A ragged batch: sequence b has rows q_start[b] .. q_start[b + 1] of the
// call's T rows, kv_len[b] cached tokens (its new ones included) and its
// pages in table[b * max_pages ..].  All on the device.
struct CacheSeqs {
  const int* q_start;
  const int* kv_len;
  const int* table;
  int T, B, max_pages;
};

struct CacheAppendArgs {
  CacheSeqs s;
  uint8_t* k;                 // e4m3 codes [pages, Hkv, page, d], pages page_stride bytes apart
  uint8_t* v;
  float* k_scale;             // [pages, Hkv]
  float* v_scale;
  int8_t* bounds;             // [pages, Hkv, 2, d] or nullptr
  long long page_stride;
  int pages, Hkv;
  const uint16_t* k_new;      // bf16 rows, k_row elements apart
  const uint16_t* v_new;
  const uint16_t* q;          // bf16 rows, or nullptr
  uint16_t* q_out;            // bf16 [T, Hq, d]
  long long k_row, v_row, q_row;
  int Hq;
  const float* rope;          // [rope_len, rope_dim]: cosines, then sines; or nullptr
  int rope_len, rope_dim, interleaved;
  DeviceStatus* status;
};

cudaError_t launch_cache_append(int page, int d, const CacheAppendArgs& a, cudaStream_t stream);

struct CacheSelectArgs {
  CacheSeqs s;
  const uint16_t* q;
  long long q_row;
  const float* k_scale;
  const int8_t* bounds;
  int pages, Hkv, group, page_shift;
  float* scores;              // workspace [T, Hkv, max_pages]
  int* selected;              // [T, Hkv, n_selected]
  int n_selected, n_first, n_recent;
  DeviceStatus* status;
};

// Whether a selection is one kernel that keeps its scores in shared memory
// (no workspace), or two with the scores between them.
bool cache_select_at_once(int max_pages);
cudaError_t launch_cache_select(int d, const CacheSelectArgs& a, cudaStream_t stream);

struct CacheAttnArgs {
  CacheSeqs s;
  const uint16_t* q;
  long long q_row;
  uint16_t* o;                // bf16 [T, Hq, d]
  float* lse;                 // [T, Hq]
  const float* k_scale;
  const float* v_scale;
  const int* selected;        // [T, Hkv, n_selected] or nullptr
  int n_selected;
  int pages, Hkv, group, page_shift, causal;
  float scale_log2;
  float* part_o;              // workspace: partial outputs of the units that CTAs share
  float2* part_ml;
  int4* rec;
  uint8_t* q_codes;           // tcgen05 kernel: queries as e4m3 pairs, hi [T * Hq, d], lo q_lo bytes further
  long long q_lo;
  float* q_scale;             // the power of two taken out of each row
  int grid;                   // CTAs of the main kernel
  DeviceStatus* status;
  long long wait_budget;
};

constexpr int kSms = 152;            // of one GB300
constexpr int kDecodeRows = 16;      // rows of a unit, keys of a piece of its work and CTAs per SM
constexpr int kDecodeKeys = 128;
constexpr int kDecodeUnitCost = 2;   // pieces that a unit counts beyond its chunks
constexpr int decode_ctas(int d) { return d == 64 ? 3 : 2; }
constexpr int kChunkRows = 256;
constexpr int kChunkTileKeys = 128;
constexpr int kChunkUnitCost = 3;
constexpr int kChunkCtas = 1;
// Rows of partial results in the workspace: two units of a CTA, `rows` each.
constexpr long long part_rows(int d, int rows) {
  return 2ll * kSms * (rows == kChunkRows ? kChunkCtas : decode_ctas(d)) * rows;
}

// Few rows per sequence (tiles of 16, mma.sync); tk, tv: 3-D uint8 views
// {d, Hkv * page, pages} of the codes, boxes of 32 rows, swizzled by a row's
// width.
cudaError_t launch_cache_decode(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CacheAttnArgs& a, cudaStream_t stream);

// Many rows per sequence (units of 256, tcgen05); tk, tv: the same views with
// boxes of one page's rows.
cudaError_t launch_cache_chunk(int d, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CacheAttnArgs& a, cudaStream_t stream);

// Joins the units of `rows` rows that CTAs of either kernel shared.
cudaError_t launch_cache_join(int d, int rows, const CacheAttnArgs& a, cudaStream_t stream);

// ------------------------------------------------------------------ paged latent cache

constexpr int kLatentRope = 64;      // columns of the rotated key part

struct LatentAppendArgs {
  CacheSeqs s;
  uint16_t* data;             // bf16 [pages, page, rank + 64], pages page_stride elements apart
  long long page_stride;
  int pages, page_shift, rank;
  const uint16_t* latent;     // bf16 rows of rank and of 64 columns
  const uint16_t* k_rope;
  long long latent_row, k_row;
  const uint16_t* q_rope;     // bf16 [T, Hq, 64], or nullptr
  long long qr_row, qr_head;
  uint16_t* q;                // bf16 [T, Hq, rank + 64]: its last 64 columns are written
  int Hq;
  const float* rope;          // [rope_len, 64] or nullptr
  int rope_len, interleaved;
  DeviceStatus* status;
};

cudaError_t launch_latent_append(const LatentAppendArgs& a, cudaStream_t stream);

struct LatentAttnArgs {
  CacheSeqs s;
  const uint16_t* data;       // bf16 [pages, page, rank + 64], pages page_stride elements apart
  long long page_stride;
  uint16_t* o;                // bf16 [T, Hq, rank]
  float* lse;                 // [T, Hq]
  int pages, page_shift, Hq, causal;
  float scale_log2;
  int span, shares;           // row blocks that work side by side, and their groups; span * shares CTAs
  float* part_o;              // workspace: partial outputs of the units that CTAs share
  float2* part_ml;
  int4* rec;
  DeviceStatus* status;
  long long wait_budget;
};

constexpr int kLatentKeys = 64;      // keys of a tile
// Tiles that a unit of so many rows a block counts beyond its own when the work is dealt:
// its queries and results.  In us with 0, 2, 3, 4: 64 sequences of 500 to 8000 keys, 16
// heads 67.3, 67.0, 67.6, 68.1, 128 heads 109, 104.7, 101.9, 100.3; 24 of 4000 keys, 128
// heads 57.3, 53.5, 51.5, 53.4; 32 of 1000 to 4000 keys, 1 to 5 tokens of 40 heads
// (rank 256) 40.5, 37.7, 37.1, 37.7.
constexpr int latent_unit_cost(int rows) { return rows < 64 ? 2 : 3; }

constexpr int kLatentPairRank = 512;   // pairs of CTAs: the latent width that they are for,
constexpr int kLatentPairRows = 128;   // rows of a unit and keys of a tile
constexpr int kLatentPairKeys = 128;

// rows: 16, 32 or 64 rows a unit; rank: 256 or 512.  tk: view {rank + 64, page, pages} of the
// cache, boxes of 64 columns and min(page, 64) rows; tq: view {64, T * Hq, rank / 64 + 1} of
// the queries by chunks of 64 columns, boxes of `rows` rows and all chunks.
cudaError_t launch_latent_attn(int rows, int rank, const CUtensorMap& tk, const CUtensorMap& tq,
                               const LatentAttnArgs& a, cudaStream_t stream);

// 128 rows a unit, on pairs of CTAs, rank 512; tq with boxes of 64 rows.
cudaError_t launch_latent_pair(const CUtensorMap& tk, const CUtensorMap& tq, const LatentAttnArgs& a,
                               cudaStream_t stream);
// Joins the units that their shares split (part of launch_latent_pair).
cudaError_t launch_latent_join_pairs(const LatentAttnArgs& a, cudaStream_t stream);

// Tensor map of bf16 data: 2 to 5 dimensions, strides of all but the first in
// elements, 128-byte swizzle (a box has 64 of the first).  Returns a fattn_status.
int make_map_bf16(CUtensorMap* m, const void* ptr, int dims, const long long* extents, const long long* strides,
                  const int* box);

// Per-device state for entry points outside fattn_api.cu: checks the device,
// gives the status word and the wait budget.  Returns a fattn_status.
int call_setup(DeviceStatus** status, long long* wait_budget);

// 3-D uint8 view {inner, rows, slabs} (rows inner bytes apart, slabs
// slab_stride), boxes of box_rows whole rows, swizzled by the row's width
// (inner 64 or 128).  Returns a fattn_status.
int make_rows_map_u8(CUtensorMap* m, const void* ptr, int inner, long long rows, int slabs,
                     long long slab_stride, int box_rows);

cudaError_t launch_selftest_timeout(DeviceStatus* status, long long budget, cudaStream_t stream);

}  // namespace fattn
