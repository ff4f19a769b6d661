/*
 * libfattn — exact, IO-aware scaled-dot-product attention for GB300 (sm_103a).
 *
 * The problem follows the pages' statement of it ("6.1 FlashAttention V1详解",
 * §8.1 tensor shapes): Q, K, V are [B, H, N, d] (batch, head, sequence,
 * head dimension); the forward pass writes O [B, H, N, d] and a per-row
 * logsumexp L [B, H, N]; the backward pass recomputes P from Q, K and L and
 * writes dQ, dK, dV.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are DEVICE pointers owned by the caller.  Tensors are
 *    dense and contiguous: bf16 [B, H, N, d] for q, k, v, o, dO, dq, dk, dv;
 *    fp32 [B, H, N] for lse.  Every pointer must be 16-byte aligned.
 *  - d is 64 or 128.  B, H, N >= 1 and B*H*N*d < 2^31.  Self-attention only
 *    (the key length equals the query length N).
 *  - scale multiplies Q K^T; it must be finite and > 0 (the usual choice is
 *    1/sqrt(d), "6.1 FlashAttention V1详解" §1.1).
 *  - causal != 0 hides key j from query i when j > i (square, top-left
 *    aligned mask).
 *  - Calls are asynchronous on `stream` (0 = legacy default stream) and
 *    return once the work is enqueued.  The library allocates no memory per
 *    call; the backward pass takes a caller-owned workspace.
 *  - Errors: argument problems return FATTN_ERR_INVALID_ARG or
 *    FATTN_ERR_UNSUPPORTED and enqueue nothing.  A failed launch returns
 *    FATTN_ERR_CUDA.  Kernels never trap: a pipeline wait that exceeds its
 *    time budget makes the kernel record FATTN_ERR_TIMEOUT in a device status
 *    word and return; fattn_check_status() reports (and clears) it.
 */
#ifndef FATTN_H_
#define FATTN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* fattn_stream_t; /* same type as cudaStream_t */

typedef enum {
  FATTN_OK = 0,
  FATTN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size or scale */
  FATTN_ERR_UNSUPPORTED = 2, /* d not in {64,128}, or the device is not sm_103 */
  FATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed */
  FATTN_ERR_TIMEOUT = 4,     /* a kernel gave up on a pipeline wait */
  FATTN_ERR_TOO_LARGE = 5,   /* the problem needs more scratch than fattn_bwd_noalloc has, or
                                fattn_cache_fwd more than 2^31 pieces of work */
  FATTN_ERR_DEBUG_CHECK = 6, /* debug builds only (FATTN_DEBUG): a kernel found an index out of
                                its range, skipped the access and recorded the site */
  FATTN_ERR_BAD_INDEX = 7,   /* a cache call's q_start, kv_len, page_table, positions or selected
                                pages are out of range; the kernel skipped what they point at */
  FATTN_ERR_NO_PAGES = 8     /* fattn_pages_extend: the pool has too few free pages; no sequence
                                was given any, and those that lack room have new_len -1 */
} fattn_status;

/*
 * Forward pass.
 * Computes S = scale * Q K^T (masked), P = softmax(S) row-wise, O = P V, and
 * L = m + log(l) per row (natural log) — "6.1 FlashAttention V1详解" §1.1 and
 * §3.2 (online softmax), "FlashAttention v1～v4" v2 §1 (L instead of m, l).
 * The N x N matrices S and P never reach device memory.
 *   q, k, v : in,  bf16 [B,H,N,d]
 *   o       : out, bf16 [B,H,N,d]
 *   lse     : out, fp32 [B,H,N]
 * Returns a fattn_status.
 */
int fattn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
              int B, int H, int N, int d, int causal, float scale,
              fattn_stream_t stream);

/*
 * FP8 forward ("FlashAttention v1～v4" v3 §3: FP8 operands with block
 * quantization).  d must be 128 (FATTN_ERR_UNSUPPORTED otherwise).
 *
 * fattn_quantize_fp8 turns a bf16 [B,H,N,d] tensor into e4m3 codes with one
 * scale per 128 consecutive rows of a head (a block):
 *   scale = amax(|x| over the block) / 448 (1 for an all-zero block),
 *   code  = e4m3(x * (1 / scale)), rounded to nearest even and saturated at
 *           +-448; the division, the reciprocal and the product are fp32.
 *   x      : in,  bf16 [B,H,N,d], 16-byte aligned
 *   codes  : out, uint8 [B,H,N,d], or with transposed != 0 uint8 [B,H,d,Np]
 *            (Np = N rounded up to 128, zero codes for rows >= N); size from
 *            fattn_fp8_codes_bytes; 16-byte aligned
 *   scales : out, fp32 [B,H,ceil(N/128)]
 * Q and K are quantized as they are, V transposed.  Returns a fattn_status.
 *
 * fattn_fwd_fp8 computes the forward pass of fattn_fwd on the dequantized
 * inputs (code value x block scale), with both GEMMs on e4m3 operands and
 * fp32 accumulation: S = sq_i sk_j (Q8 K8^T); the probabilities of key block
 * j are multiplied by sv_j / max_j' sv_j' (at most 1) and rounded to e4m3 for
 * P V, and O is rescaled once at the end; the row sums behind O's
 * normalisation and L use the fp32 probabilities.
 *   q8, k8  : in, uint8 [B,H,N,d] codes;   sq, sk: in, fp32 [B,H,ceil(N/128)]
 *   v8t     : in, uint8 [B,H,d,Np] codes;  sv: in, fp32 [B,H,ceil(N/128)]
 *   o, lse  : out, as for fattn_fwd
 * Returns a fattn_status.
 */
size_t fattn_fp8_codes_bytes(int B, int H, int N, int d, int transposed);
int fattn_quantize_fp8(const void* x, void* codes, float* scales, int B, int H, int N, int d,
                       int transposed, fattn_stream_t stream);

/*
 * Incoherent processing ("FlashAttention v1～v4" v3 §3): quantize x M instead
 * of x, M = diag(signs) H / sqrt(d) with H the Sylvester-Hadamard matrix, an
 * orthogonal matrix, so quantizing Q M and K M leaves S = Q K^T unchanged in
 * exact arithmetic while an outlier's energy is spread over all d columns
 * before the block scale is taken.  Each row is rotated in fp32 (the signs,
 * butterflies a + b / a - b at strides 1, 2, ..., 64, then one multiplication
 * by fp32(1/sqrt(d))), then quantized as by fattn_quantize_fp8 (not
 * transposed).  Apply it to Q and K with the same signs, never to V.
 *   signs : in, fp32 [d] of +1 / -1, 16-byte aligned (only the sign bit of
 *           each entry is read)
 * Other arguments as for fattn_quantize_fp8; d must be 128.
 */
int fattn_quantize_fp8_rotated(const void* x, const float* signs, void* codes, float* scales,
                               int B, int H, int N, int d, fattn_stream_t stream);
int fattn_fwd_fp8(const void* q8, const float* sq, const void* k8, const float* sk,
                  const void* v8t, const float* sv, void* o, float* lse, int B, int H, int N,
                  int d, int causal, float scale, fattn_stream_t stream);

/*
 * Backward preprocessing: D_i = sum_k dO_ik * O_ik (fp32, one value per row;
 * the identity rowsum(dP o P) = rowsum(dO o O) of "6.1 FlashAttention
 * V1详解" §6.1), and zero the fp32 dQ accumulator.
 *   o, dO    : in,  bf16 [B,H,N,d]
 *   D        : out, fp32 [B,H,N]
 *   dq_accum : out, fp32 [B,H,N,d], set to zero
 * fattn_bwd runs this itself; it is exported for callers that schedule it.
 */
int fattn_bwd_preprocess(const void* o, const void* dO, float* D, float* dq_accum,
                         int B, int H, int N, int d, fattn_stream_t stream);

/*
 * Workspace the backward pass needs, in bytes: D and -L*log2(e) (fp32, each
 * [B*H, Np] with Np = N rounded up to a multiple of 128), then the fp32 dQ
 * accumulator ([B,H,N,d]), then one uint32 dQ contribution counter per head
 * and 128-row Q tile ([B*H, Np/128], used in deterministic mode); each part
 * starts on a 256-byte boundary.  Returns 0 for invalid sizes.
 */
size_t fattn_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward pass ("6.1 FlashAttention V1详解" §6.1-6.2, recomputation):
 * P is rebuilt from Q, K and L; then dV = P^T dO, dP = dO V^T,
 * dS = P o (dP - D), dQ = scale dS K, dK = scale dS^T Q (the last two by
 * the chain rule through S = scale Q K^T).
 *   q, k, v, o, dO : in,  bf16 [B,H,N,d];  lse: in, fp32 [B,H,N] from fattn_fwd
 *   dq, dk, dv     : out, bf16 [B,H,N,d]
 *   workspace      : scratch of at least fattn_bwd_workspace_bytes(B,H,N,d),
 *                    256-byte aligned, caller-owned; contents on entry ignored
 * Enqueues, in order: preprocess, the main backward kernel (dQ accumulated
 * with fp32 reduce-adds, in a fixed order when fattn_set_deterministic is on),
 * and the dQ conversion.  Returns a fattn_status.
 */
int fattn_bwd(const void* q, const void* k, const void* v, const void* o,
              const void* dO, const float* lse, void* dq, void* dk, void* dv,
              void* workspace, size_t workspace_bytes,
              int B, int H, int N, int d, int causal, float scale,
              fattn_stream_t stream);

/*
 * The three stages that fattn_bwd enqueues, exported for callers that time
 * or schedule them separately.  Run in this order on one workspace they do
 * exactly what fattn_bwd does:
 *   fattn_bwd_prepare: D = rowsum(dO o O) and -L*log2(e) into the workspace,
 *                      and zero its fp32 dQ accumulator;
 *   fattn_bwd_main:    the recomputation kernel: writes dk, dv and adds the
 *                      dQ partial sums into the accumulator;
 *   fattn_bwd_finish:  dq = bf16(scale * accumulator).
 * Arguments have the meaning given for fattn_bwd; the workspace must hold at
 * least fattn_bwd_workspace_bytes(B,H,N,d) bytes, 256-byte aligned.
 */
int fattn_bwd_prepare(const void* o, const void* dO, const float* lse,
                      void* workspace, size_t workspace_bytes,
                      int B, int H, int N, int d, fattn_stream_t stream);
int fattn_bwd_main(const void* q, const void* k, const void* v, const void* dO,
                   void* workspace, size_t workspace_bytes, void* dk, void* dv,
                   int B, int H, int N, int d, int causal, float scale,
                   fattn_stream_t stream);
int fattn_bwd_finish(const void* workspace, size_t workspace_bytes, void* dq,
                     int B, int H, int N, int d, float scale, fattn_stream_t stream);

/* Size of the scratch array built into the library for fattn_bwd_noalloc. */
#define FATTN_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/*
 * Backward pass for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this entry point; it is a service of the
 * library.  It does what fattn_bwd does, with the same arguments minus the
 * workspace, but takes its scratch (D, -L*log2(e) and the fp32 dQ
 * accumulator) from a fixed device array compiled into the library
 * (FATTN_NOALLOC_SCRATCH_BYTES, 64 MiB, held on every device that loads the
 * library until the process exits).  It is meant for code that has no way
 * to obtain device memory at the point of the call: a plugin whose host
 * framework owns every allocation and forbids the plugin to make its own,
 * a real-time loop in which cudaMalloc's implicit device synchronisation is
 * not acceptable, or a caller that simply has no spare buffer to pass.
 * This call itself never calls cudaMalloc, cudaFree or any allocating
 * routine.
 *
 *  - Size limit: fattn_bwd_workspace_bytes(B,H,N,d) must not exceed
 *    FATTN_NOALLOC_SCRATCH_BYTES (about B*H*N <= 127,000 at d = 128 and
 *    <= 250,000 at d = 64); larger problems return FATTN_ERR_TOO_LARGE and
 *    enqueue nothing.
 *  - The first call on a device looks up the array's device address (no
 *    allocation); make that first call before any stream capture begins.
 *  - Every call on a device uses the same array, and the array keeps the
 *    last call's contents; the call re-initialises everything it reads.
 *    Calls whose work overlaps on the GPU (other streams, other host
 *    threads) race on the array: serialise them.
 * Returns a fattn_status.
 */
int fattn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                      const void* dO, const float* lse, void* dq, void* dk, void* dv,
                      int B, int H, int N, int d, int causal, float scale,
                      fattn_stream_t stream);

/*
 * The static work schedule of the backward's main kernel, computed on the
 * host (no GPU, no CUDA call, nothing enqueued).  A work item is the 128-row
 * K/V tile j of head bh = b*H + h, which walks its Q tiles (causal: tiles
 * j..n_tiles-1; n_tiles = ceil(N/128)); the kernel runs one CTA per SM, each
 * working through a list of items fixed before the launch ("FlashAttention
 * v1～v4" v4 §4: persistent scheduling, heaviest first, L2-aware head order).
 *   B, H, N, d    : as for fattn_bwd_main; causal, deterministic as there
 *                   (deterministic = the mode of fattn_set_deterministic)
 *   grid          : number of CTAs; a launch uses min(SM count, B*H*n_tiles)
 *   l2_bytes      : L2 size the head sections are sized for
 *                   (cudaDevAttrL2CacheSize on the device)
 *   item_cta      : out, int [B*H*n_tiles], caller-owned host memory: at
 *                   [bh*n_tiles + j] the CTA that processes K/V tile j of head
 *                   bh; -1 if no CTA does, -2 if several do (neither happens)
 *   cta_q_tiles   : out, optional (NULL), long long [grid], host memory: the
 *                   Q tiles each CTA walks, i.e. its share of the work
 * Returns FATTN_ERR_INVALID_ARG for bad sizes, grid < 1, grid above the item
 * count, more than 2^24 items or a NULL item_cta; FATTN_ERR_UNSUPPORTED for
 * d not in {64, 128}.
 */
int fattn_bwd_schedule(int B, int H, int N, int d, int causal, int deterministic, int grid,
                       long long l2_bytes, int* item_cta, long long* cta_q_tiles);

/*
 * The same schedule in processing order, for checking it on the host (no
 * GPU): every CTA's work items in the order it runs them, with the Q tiles
 * each item visits.  The ordered dQ reduction of the deterministic mode
 * waits, at every Q tile, for the smaller K/V tiles of the head; whether
 * such a schedule can always make progress is a property of this order.
 *   B .. l2_bytes : as for fattn_bwd_schedule
 *   cta_start     : out, int [grid + 1], host memory: CTA c's items are
 *                   entries cta_start[c] .. cta_start[c + 1] - 1 of items
 *   items         : out, int [5 * B*H*n_tiles], host memory: per entry
 *                   (bh, j, i0, n_it, rot); step it of the item visits Q tile
 *                   i0 + it when causal, (rot + it) mod n_tiles otherwise
 * Returns as fattn_bwd_schedule (NULL cta_start or items: invalid).
 */
int fattn_bwd_schedule_items(int B, int H, int N, int d, int causal, int deterministic, int grid,
                             long long l2_bytes, int* cta_start, int* items);

/*
 * The schedule of the CTA-pair backward (fattn_set_bwd_pair; d = 128), on
 * the host: per cluster of two CTAs, its work units in processing order.  A
 * unit is K/V tiles 2u (rank 0) and 2u + 1 (rank 1) of one head.
 *   B, H, N, causal, l2_bytes : as for fattn_bwd_schedule
 *   clusters      : number of CTA pairs of the launch
 *   cluster_start : out, int [clusters + 1]: cluster c's units are entries
 *                   cluster_start[c] .. cluster_start[c + 1] - 1 of items
 *   items         : out, int [5 * B*H*ceil(ceil(N/128)/2)]: per entry
 *                   (bh, 2u, i0, n_it, rot), visiting Q tiles as in
 *                   fattn_bwd_schedule_items
 * Returns FATTN_ERR_INVALID_ARG for bad sizes, clusters < 1 or above the
 * unit count, more than 2^24 units, or NULL outputs.
 */
int fattn_bwd_pair_schedule_items(int B, int H, int N, int causal, int clusters, long long l2_bytes,
                                  int* cluster_start, int* items);

/*
 * Attention over a paged 8-bit cache
 * ----------------------------------
 * Answering token by token needs the keys and values of earlier tokens.  The
 * pages have no counterpart to these entry points; they carry the FP8
 * forward's block quantization to a cache that the caller owns.  Keys and
 * values are e4m3 codes with one scale per page and kv head:
 *   k, v             : uint8 [pages, Hkv, page, d], contiguous within a page; the pages of
 *                      both lie page_stride bytes apart (at least Hkv*page*d, a multiple of 16);
 *                      16-byte aligned
 *   k_scale, v_scale : fp32 [pages, Hkv], each a power of two 2^e, -48 <= e <= 48; a value is
 *                      code * scale
 *   k_bounds         : int8 [pages, Hkv, 2, d] or NULL: per column the lower and the upper bound
 *                      of the page's key codes in units of 448/127 of the scale (for
 *                      fattn_cache_select); 16-byte aligned
 *   page             : 32, 64 or 128 tokens;  d: 64 or 128;  Hkv <= 1024
 *
 * A call works on a ragged batch of B <= 4096 sequences, described on the
 * device so that a captured graph can be replayed on other lengths:
 *   q_start    : int [B+1], ascending; rows q_start[b] .. q_start[b+1]-1 of the call's T rows are
 *                the new tokens of sequence b (none is allowed).  Rows from q_start[B] on are
 *                padding: nothing of theirs is read or written.
 *   kv_len     : int [B], the tokens of sequence b in the cache, its new ones included; the last
 *                n_b = q_start[b+1]-q_start[b] of them are the new ones, so row i of the sequence
 *                has position kv_len[b] - n_b + i
 *   page_table : int [B, max_pages]; token t of sequence b is slot t % page of page
 *                page_table[b][t / page]; entries past ceil(kv_len/page) are not read
 * Query head h belongs to kv head h / (Hq / Hkv); Hkv divides Hq, Hq / Hkv <= 128.  Rows of
 * q, k_new and v_new may lie further apart than they are long (slices of one projection):
 * q_row, k_row, v_row are their distances in elements, multiples of 8.
 * The kernels check these numbers before they use them: a sequence with
 * senseless q_start or kv_len counts as empty, tokens on a page outside the cache count as
 * absent, and fattn_check_status() reports FATTN_ERR_BAD_INDEX.
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  void* k_bounds;
  long long page_stride;
  int pages, Hkv, page, d;
} fattn_cache;

/*
 * Append the batch's new tokens to the cache, keys rotated by their positions.
 * Rotation: with rope = fp32 [rope_len, rope_dim], row p the rope_dim/2
 * cosines of position p's angles and then the sines, column pairs (a, b) of a
 * head become (a cos - b sin, b cos + a sin); the pairs are columns (i,
 * i + rope_dim/2), or (2i, 2i+1) when interleaved != 0; columns from rope_dim on
 * stay.  rope_dim is a multiple of 16 up to d; rope NULL (rope_dim 0) rotates
 * nothing.  fp32, every product and sum rounded.
 * Quantization: a page and head has scale 2^e with e the smallest exponent in
 * [-48, 48] for which amax <= 448 * 2^e over its tokens, or the exponent it has if that is
 * larger; code = e4m3(x * 2^-e), nearest even, saturated (so an infinity becomes
 * 448 * 2^48, which leaves nothing of its page's other tokens).  When new tokens
 * raise e, the page's earlier codes are multiplied by the power of two and
 * rounded again.  A page whose slot 0 is among the new tokens starts over.
 * A token with a NaN in a head's key or value gets a NaN key and a zero
 * value: the rows that attend to it become NaN, and no others.
 *   k_new, v_new : in, bf16 rows of Hkv*d
 *   q, q_out     : in, bf16 rows of Hq*d, and out, bf16 [T, Hq, d]: the queries rotated likewise
 *                  (q_out may be q when its rows are contiguous); both NULL: none
 * A page that receives tokens must belong to one sequence only.  Positions
 * below 0 or from rope_len on are FATTN_ERR_BAD_INDEX; of a sequence that has
 * any, nothing is appended and no query written.  Returns a fattn_status.
 */
int fattn_cache_append(const fattn_cache* cache, const void* k_new, long long k_row,
                       const void* v_new, long long v_row, const void* q, long long q_row,
                       void* q_out, int Hq, const float* rope, int rope_len, int rope_dim,
                       int interleaved, const int* page_table, const int* q_start,
                       const int* kv_len, int T, int B, int max_pages, fattn_stream_t stream);

/*
 * Attention of the batch's rows over their sequences' cached tokens.  Row i
 * sees the tokens before position kv_len, and with causal != 0 those up to its
 * own position; a row that sees nothing gets O = 0 and L = -inf, and one that
 * sees a key and has an infinity or a NaN in its query becomes NaN.
 *   q          : in,  bf16 rows of Hq*d (rotated)
 *   o, lse     : out, bf16 [T, Hq, d] and fp32 [T, Hq], as for fattn_fwd
 *   selected   : in, int [T, Hkv, n_selected] or NULL (n_selected 0): row t's heads of kv head h
 *                attend only to the pages page_table[b][selected[t][h][i]] of their sequence;
 *                negative entries stand for none, an entry named twice counts twice
 *   workspace  : at least fattn_cache_fwd_workspace_bytes(T, B, Hq, Hkv, d, n_selected) bytes,
 *                256-byte aligned; contents on entry ignored; calls that may overlap need
 *                one each
 * Value slots behind a sequence's end may hold anything; those before it hold
 * no NaN code (fattn_cache_append writes none).
 * Rounding: a query enters the products off by at most 2^-17 of its row's
 * largest entry (exact for entries above 2^-9 of it), probabilities are rounded
 * to fp16 (2^-11) for P V, and O to bf16 (2^-8); scores, sums, maxima and the
 * accumulators are fp32.
 * One of two kernels, for few and for many rows, serves the whole call.  The
 * choice goes by the rows of an average sequence, T * (Hq / Hkv) / B, and for 17 to 64
 * of them also by min(B * max_pages, pages), as the lengths are on the device.
 * Selected pages go to the one for few rows.  Both are right for every batch;
 * their results may differ in the last bits.  A batch that mixes pieces of
 * prompts with many single tokens is faster as two calls.
 * Results do not depend on timing.  Returns a fattn_status.
 */
size_t fattn_cache_fwd_workspace_bytes(int T, int B, int Hq, int Hkv, int d, int n_selected);
int fattn_cache_fwd(const fattn_cache* cache, const void* q, long long q_row, void* o, float* lse,
                    const int* page_table, const int* q_start, const int* kv_len,
                    const int* selected, int n_selected, void* workspace, size_t workspace_bytes,
                    int T, int B, int Hq, int max_pages, int causal, float scale,
                    fattn_stream_t stream);

/*
 * Choose, for each row and kv head, the n_selected pages of the row's
 * sequence that matter most, by an upper bound of the sum of the group's
 * scores from the cache's k_bounds:
 *   q8 = round(q * (127 / amax)), amax over the group's Hq/Hkv * d entries (fp32; zero below 2^-100),
 *   score(page) = float(sum_d (sum_h max(q8,0)) hi_d + (sum_h min(q8,0)) lo_d) * k_scale,
 * the sums in whole numbers, so the choice is exact.  The first n_first pages
 * and the last n_recent up to the row's own are always taken (n_first + n_recent <= n_selected); ties go to
 * the lower page.  A row with no more than n_selected pages takes them all.
 *   q         : in,  bf16 rows of Hq*d, as for fattn_cache_fwd
 *   selected  : out, int [T, Hkv, n_selected]: ascending, -1 behind the last
 *   workspace : at least fattn_cache_select_workspace_bytes(T, Hkv, max_pages), 256-byte aligned;
 *               contents on entry ignored; NULL (0 bytes) will do where that function says 256, the
 *               sizes that keep their scores on chip
 * max_pages is at most 65535 * 128 here.  Returns a fattn_status.
 */
size_t fattn_cache_select_workspace_bytes(int T, int Hkv, int max_pages);
int fattn_cache_select(const fattn_cache* cache, const void* q, long long q_row,
                       const int* page_table, const int* q_start, const int* kv_len,
                       int* selected, int n_selected, int n_first, int n_recent, void* workspace,
                       size_t workspace_bytes, int T, int B, int Hq, int max_pages,
                       fattn_stream_t stream);

/*
 * Rotary positions
 * ----------------
 * y = x with the pairs of each row's first rope_dim columns rotated by the angles
 * of the row's position, (a cos - b sin, b cos + a sin); the other columns stay.  With
 * transposed != 0 by the negated angles: the gradient, dx = R^T dy.  Pairs, the
 * table (fp32 [rope_len, rope_dim]) and the arithmetic (fp32, every product and sum
 * rounded, then one rounding to bf16) are those of fattn_cache_append.
 *   x, y       : bf16 rows of d columns, row (b, h, n) of [B, H, N, d] at b x_b + h x_h + n x_n
 *                elements; these are multiples of 8 from 0 (x only) up to 2^40, and rows
 *                of y do not overlap.  y may be x with the same distances, and then only the
 *                rotated columns are touched; otherwise they share no element.  d is a multiple
 *                of 16 up to 1024 (FATTN_ERR_UNSUPPORTED)
 *   positions  : int, row (b, n) at positions[b * positions_b + n] (0: the same for all b), or
 *                NULL: n.  Rows whose position is outside [0, rope_len) are not written
 *                and are FATTN_ERR_BAD_INDEX
 * rope_dim is a multiple of 16 up to d.  Returns a fattn_status.
 */
int fattn_rope(const void* x, long long x_b, long long x_h, long long x_n, void* y, long long y_b,
               long long y_h, long long y_n, const float* rope, int rope_len, int rope_dim,
               int interleaved, int transposed, const int* positions, long long positions_b, int B,
               int H, int N, int d, fattn_stream_t stream);

/*
 * Attention over a paged latent cache
 * -----------------------------------
 * Where the keys and values of all heads are products of one latent vector a token,
 * the cache holds that vector and the token's rotated key part, which the heads
 * share, and queries come multiplied with the keys' product (the absorbed form):
 *   data  : bf16 [pages, page, rank + 64], contiguous within a page, the pages page_stride
 *           elements apart (a multiple of 8, below 2^38); 16-byte aligned.  Columns 0 .. rank-1 are a
 *           token's latent, its value for every head; all columns are its key
 *   rank  : 256 or 512;  page: 32, 64 or 128 tokens
 * The batch is described as for fattn_cache_fwd: q_start, kv_len, page_table, checked
 * by the kernels.  Query heads: Hq <= 1024.
 */
typedef struct {
  void* data;
  long long page_stride;
  int pages, page, rank;
} fattn_latent_cache;

/*
 * Append the batch's new tokens: latents as they are, key parts rotated by their
 * positions (as in fattn_cache_append, rope_dim 64; rope NULL rotates nothing), and
 * the queries' parts likewise.
 *   latent  : in, bf16 rows of rank columns, latent_row elements apart
 *   k_rope  : in, bf16 rows of 64 columns, k_row apart (both multiples of 8: slices of
 *             one projection)
 *   q_rope  : in, bf16 [T, Hq, 64], rows q_row and heads q_head elements apart (multiples of 8)
 *   q       : out, bf16 [T, Hq, rank + 64], contiguous: columns rank .. rank+63 are written.
 *             q_rope and q may be the same columns of one buffer; both NULL: none
 * A token with an infinity or a NaN in its latent or key part gets a NaN key part
 * and a zero latent: the rows that attend to it become NaN, and no others.
 * A page that receives tokens must belong to one sequence only.  Positions below 0 or
 * from rope_len on are FATTN_ERR_BAD_INDEX; of a sequence that has any, nothing is
 * appended and no query written.  Returns a fattn_status.
 */
int fattn_latent_append(const fattn_latent_cache* cache, const void* latent, long long latent_row,
                        const void* k_rope, long long k_row, const void* q_rope, long long q_row,
                        long long q_head, void* q, int Hq, const float* rope, int rope_len,
                        int interleaved, const int* page_table, const int* q_start,
                        const int* kv_len, int T, int B, int max_pages, fattn_stream_t stream);

/*
 * Attention of the batch's rows over their sequences' cached tokens: with c_j the
 * latent and k_j all columns of token j,
 *   s_j = scale q . k_j,  O = sum_j softmax(s)_j c_j,  L = log sum_j exp(s_j)
 * per row and head.  Masks, rows that see nothing and queries with an infinity or a
 * NaN as in fattn_cache_fwd.
 *   q         : in,  bf16 [T, Hq, rank + 64], contiguous
 *   o, lse    : out, bf16 [T, Hq, rank] and fp32 [T, Hq]
 *   workspace : at least fattn_latent_fwd_workspace_bytes(T, B, Hq, rank) bytes, 256-byte
 *               aligned; contents on entry ignored; calls that may overlap need one each
 * Slots behind a sequence's end may hold anything; latents before it are finite
 * (fattn_latent_append writes no others).
 * Rounding: probabilities are rounded to bf16 (2^-8) for the second product, and O to
 * bf16 (2^-8); scores, sums, maxima and the accumulators are fp32.  O is divided by the sum
 * of the rounded probabilities, so that its weights add up to one; L is of the others.
 * The rows of an average sequence, T * Hq / B, and for more than 64 of them the room of the
 * tables, max_pages * page, decide how the call is laid out (sums are then taken in another
 * order); a batch that mixes pieces of prompts with many single tokens is faster as two
 * calls.  Results do not depend on timing.  Returns a fattn_status.
 */
size_t fattn_latent_fwd_workspace_bytes(int T, int B, int Hq, int rank);
int fattn_latent_fwd(const fattn_latent_cache* cache, const void* q, void* o, float* lse,
                     const int* page_table, const int* q_start, const int* kv_len, void* workspace,
                     size_t workspace_bytes, int T, int B, int Hq, int max_pages, int causal,
                     float scale, fattn_stream_t stream);

/*
 * The pages of a cache
 * --------------------
 * Sequences may share pages (a prompt and its samples).  A pool counts, on the device, how
 * many table entries name each page, so that pages can be taken, shared and given back
 * between the steps of a captured graph:
 *   refs  : int [pages], zeros for an empty pool; a page is free while its count is 0
 *   page  : 32, 64 or 128 tokens;  pages < 2^30
 * Sequence b holds the first ceil(len/page) entries of its row of page_table [B, max_pages];
 * the others are neither read nor written.  B <= 4096.  The lowest free pages are taken
 * first, so results do not depend on timing.
 *
 * A cache is any number of planes (at most 5), page p of each at base + p * stride bytes:
 * bytes, stride and base are multiples of 4 (of 16 for wide copies).  A
 * fattn_cache has k, v, k_scale, v_scale and k_bounds, a fattn_latent_cache one.
 */
typedef struct {
  int* refs;
  int pages, page;
} fattn_page_pool;

typedef struct {
  void* base;
  long long stride, bytes;
} fattn_plane;

/*
 * Sequence child[i] becomes a copy of sequence parent[i] that shares its pages: its table
 * entries, its length (kv_len, in and out), and one more count for each of its pages.
 *   parent, child : int [n] on the device, n <= B.  A child has length 0 before; one that has not, is
 *                   named twice, is out of range or is also a parent is
 *                   FATTN_ERR_BAD_INDEX and left as it is
 * Returns a fattn_status.
 */
int fattn_pages_fork(const fattn_page_pool* pool, int* page_table, int* kv_len, const int* parent,
                     const int* child, int n, int B, int max_pages, fattn_stream_t stream);

/*
 * Make room for the tokens old_len[b] .. new_len[b]-1 of every sequence, to be called
 * before they are appended.  In order of b: where token old_len[b] falls into a page that it
 * shares, the sequence gets a copy of that page for itself (the last that still has the
 * page keeps it), and then the pages it lacks.
 *   old_len, new_len : int [B] on the device, 0 <= old_len <= new_len <= max_pages * page; a
 *                      sequence with others is FATTN_ERR_BAD_INDEX and gets nothing.  new_len
 *                      is in and out: -1 for a sequence without room for its tokens
 *   workspace        : at least fattn_pages_workspace_bytes(pages, B), 256-byte aligned; contents on
 *                      entry ignored; calls that may overlap need one each
 * With too few free pages no sequence gets any: tables and counts stay as they are, but
 * that the entries to be filled become -1, and fattn_check_status() reports
 * FATTN_ERR_NO_PAGES.  A sequence that needed a page, or would write into one that it shares,
 * has new_len -1 then; its length is still old_len.  Append and attention, given new_len as their
 * kv_len, leave it alone (FATTN_ERR_BAD_INDEX, which the first error hides) and serve
 * the others, also in a captured step, where the host cannot look in between.  Returns a
 * fattn_status.
 */
size_t fattn_pages_workspace_bytes(int pages, int B);
int fattn_pages_extend(const fattn_page_pool* pool, const fattn_plane* planes, int n_planes,
                       int* page_table, const int* old_len, int* new_len, void* workspace,
                       size_t workspace_bytes, int B, int max_pages, fattn_stream_t stream);

/*
 * The sequences rows[i] (int [n] on the device, n <= 4096) give their pages back: one
 * count less for each, and length 0 (kv_len, in and out).  Of a row named twice the
 * first counts; a row out of range, or a page that was free already, is FATTN_ERR_BAD_INDEX.
 * Returns a fattn_status.
 */
int fattn_pages_free(const fattn_page_pool* pool, int* page_table, int* kv_len, const int* rows,
                     int n, int B, int max_pages, fattn_stream_t stream);

/*
 * Move the pool's pages together: with U pages held, the k-th held page from U on goes to the
 * k-th free page below U, in every plane, count and table entry.  kv_len [B] says which
 * entries sequences hold (pages taken for tokens beyond it would be lost: give the
 * lengths that fattn_pages_extend was given).  With a length out of range nothing moves; an
 * entry that names a page outside the pool, or one that was free, stays (both
 * FATTN_ERR_BAD_INDEX).  Workspace as for fattn_pages_extend.  Returns a fattn_status.
 */
int fattn_pages_compact(const fattn_page_pool* pool, const fattn_plane* planes, int n_planes,
                        int* page_table, const int* kv_len, void* workspace, size_t workspace_bytes,
                        int B, int max_pages, fattn_stream_t stream);

/*
 * Synchronise `stream`, then report the first error since the last call:
 * a pending asynchronous CUDA error (FATTN_ERR_CUDA), a kernel wait timeout
 * (FATTN_ERR_TIMEOUT), an index that a cache call found out of range
 * (FATTN_ERR_BAD_INDEX) or a pool without enough free pages (FATTN_ERR_NO_PAGES)
 * recorded on the current device.  Clears the
 * device status word.  Returns FATTN_OK when neither happened.
 */
int fattn_check_status(fattn_stream_t stream);

/* Static, human-readable name of a status code. */
const char* fattn_status_string(int status);

/*
 * Budget, in SM clock cycles, for every pipeline wait inside the kernels
 * (default 2^31, about one second).  Values <= 0 restore the default.
 * What a kernel has started itself it sees end, whatever the budget: copies
 * and products in flight are given 2^31 cycles.
 * Applies to launches made after the call, from any thread.
 */
void fattn_set_wait_budget(long long cycles);

/*
 * Deterministic backward ("FlashAttention v1～v4" v4 §4: cross-CTA
 * reductions in a fixed order through semaphores).  When on, every 128-row
 * tile of the fp32 dQ accumulator receives the contributions of the K/V tiles
 * in ascending tile order: the CTA holding K/V tile j waits (bounded by the
 * wait budget; a wait that runs out is a FATTN_ERR_TIMEOUT) until the
 * workspace counter of the Q tile says that tiles 0..j-1 have been added,
 * adds its own, waits for its adds to complete and advances the counter.
 * dQ, dK and dV are then bitwise identical from run to run for the same
 * inputs and device (dK and dV always are).  Off by default: dQ is otherwise
 * summed in arrival order, which differs run to run within fp32 rounding.
 * Applies to backward launches made after the call, from any thread.
 */
void fattn_set_deterministic(int on);

/*
 * Backward main kernel variant for d = 128 in the default (any-order dQ)
 * mode ("FlashAttention v1～v4" v4 §4, backward with two cooperating CTAs).
 * On: pairs of CTAs on two SMs issue every matrix product of the backward
 * together (M = 256 tiles, each CTA staging half of operand B), exchange
 * half of dS through distributed shared memory and reduce-add dQ summed
 * over both CTAs' keys.  Off (the default): one CTA per K/V tile, which
 * measures faster on GB300 (the pair's per-step hand-offs between SMs cost
 * more than the shared-memory traffic they save).  Both give the same
 * gradients up to fp32 summation order.  d = 64 and the deterministic mode
 * always use one CTA per tile.  Applies to later launches.
 */
void fattn_set_bwd_pair(int on);

/*
 * Threshold, in log2 units, of the conditional rescaling in the forward pass
 * ("FlashAttention v1～v4" v4 §3): the reference max of a row moves only when
 * the row max exceeds it by more than tau_log2, and O, l are rescaled only
 * then.  The result is exact for any tau_log2 >= 0 because l and O always
 * share the reference; probabilities stay <= 2^tau_log2.  Default 8
 * (log2 256, the page's value).  Negative values restore the default;
 * values above 16 are clamped to 16.  The FP8 forward uses at most 8: its
 * probabilities are rounded to e4m3, which saturates at 448 = 2^8.81, so a
 * larger threshold would clip them.  Applies to later launches.
 */
void fattn_set_rescale_threshold(float tau_log2);

/*
 * Self-test of the timeout path: launches one block that waits, with the
 * given cycle budget, on a barrier that nothing ever completes.  The wait
 * gives up, records FATTN_ERR_TIMEOUT in the status word and the kernel
 * returns; the next fattn_check_status() reports it.  Returns FATTN_OK if
 * the launch was enqueued.
 */
int fattn_selftest_timeout(long long budget_cycles, fattn_stream_t stream);

/* Library version, "major.minor.patch". */
const char* fattn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FATTN_H_ */
