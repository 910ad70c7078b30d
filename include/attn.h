/*
 * attn.h - C ABI of libattn.so: exact, IO-aware tiled attention on GB300 (sm_103a).
 *
 * The operation is scaled-dot-product attention, O = softmax(Q K^T / sqrt(d)) V
 * ("FlashAttention/es", section "Por qué la atención estándar es lenta"), computed
 * exactly with the tiled online-softmax recurrence ("El truco del softmax en línea"
 * and "El algoritmo FlashAttention" on the same page) so that no N x N matrix ever
 * reaches device memory. The forward pass also writes the per-row log-sum-exp
 * L_i = m_i + log(l_i) (natural log) that the backward pass uses to rebuild P
 * ("Paso hacia atrás y recomputación", same page).
 *
 * Attention variants follow the FlexAttention list in "El FlexAttention de PyTorch
 * con FlashAttention-4 es un cambio radical" (first section): score modifications
 * ALiBi and tanh soft-capping, mask modifications causal, sliding window and
 * document masking; tiles in which the mask allows nothing are skipped.
 *
 * Conventions shared by every call:
 *   - Tensors are DEVICE pointers owned by the caller, contiguous, row-major:
 *       q, o, dout, dq : bf16 [B, Hq,  Nq,  d]   (d fastest)
 *       k, v, dk, dv   : bf16 [B, Hkv, Nkv, d]
 *       lse            : fp32 [B, Hq, Nq]
 *     Every tensor pointer must be 16-byte aligned (ATTN_ERR_ALIGN otherwise).
 *   - Query head h reads kv head h / (Hq / Hkv) (grouped-query attention).
 *   - d must be 64, 128 or 256 ("FlashAttention/es", "Limitaciones": head sizes up to
 *     about 256); the SIMT entry points, the FP8 forward and dropout take 64 and 128
 *     only. Hq must be a multiple of Hkv.
 *   - scale multiplies Q K^T (usually 1/sqrt(d)); it must be finite.
 *   - Scores are modified in the order: scale, ALiBi, soft-cap, mask.
 *       ALiBi:    s_ij -= slope_h * (i - j), slope_h = 2^(-8 (h+1) / Hq),
 *                 h the 0-based query head.
 *       soft-cap: s_ij  = c * tanh(s_ij / c), c = attn_score_params.softcap > 0.
 *   - Masks (i = query position, j = key position, both from 0):
 *       ATTN_MASK_NONE               every pair
 *       ATTN_MASK_CAUSAL             j <= i (top-left aligned, also when Nq != Nkv)
 *       ATTN_MASK_SLIDING_WINDOW     j <= i and i - j < window (window >= 0;
 *                                    window 0 masks every pair)
 *       ATTN_MASK_DOCUMENT_CAUSAL    doc(i) == doc(j) and j <= i, with documents
 *                                    given by int32 DEVICE offsets
 *                                    doc_offsets[0..n_docs]: doc_offsets[0] = 0,
 *                                    non-decreasing, doc_offsets[n_docs] = Nq = Nkv.
 *                                    The offsets are trusted (not read on the host);
 *                                    attn_check_doc_offsets checks a table, and the
 *                                    checked mode (ATTN_CHECKED, below) checks it in
 *                                    every call.
 *     A query row with no allowed key gets O = 0 and lse = -inf, and zero gradients.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream). They allocate no device memory; the backward pass takes a
 *     caller-provided workspace. Results are deterministic: the same inputs give
 *     bitwise-identical outputs.
 *   - Errors are returned, never hidden: there is no fallback path. A call that
 *     returns an error launched nothing.
 *   - Sizes of 0 (B, heads, Nq or Nkv) are valid; Nkv = 0 gives masked rows.
 */
#ifndef EXACT_IO_AWARE_ATTN_H
#define EXACT_IO_AWARE_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_ARG = 1,            /* null pointer, unknown kind, bad scale/window/softcap */
  ATTN_ERR_SHAPE = 2,          /* unsupported d (256 on the SIMT/FP8 paths), Hq % Hkv != 0, negative size,
                                  document mask with Nq != Nkv, size over 2^31 */
  ATTN_ERR_ALIGN = 3,          /* a tensor pointer is not 16-byte aligned */
  ATTN_ERR_ARCH = 4,           /* the current device is not compute capability 10.3 */
  ATTN_ERR_WORKSPACE = 5,      /* workspace NULL or smaller than attn_bwd_workspace_size */
  ATTN_ERR_LAUNCH = 6,         /* a CUDA runtime/driver call or a launch failed */
  ATTN_ERR_DEVICE_TIMEOUT = 7, /* a kernel's bounded wait expired (attn_device_status) */
  ATTN_ERR_DEVICE_INPUT = 8    /* a kernel met an out-of-range DEVICE input: a decode
                                  sequence length or page index (attn_device_status) */
} attn_status;

enum {
  ATTN_MASK_NONE = 0,
  ATTN_MASK_CAUSAL = 1,
  ATTN_MASK_SLIDING_WINDOW = 2,
  ATTN_MASK_DOCUMENT_CAUSAL = 3
};

/* Score modification flags (OR-able; ALiBi is applied before soft-cap). */
enum {
  ATTN_SCORE_NONE = 0,
  ATTN_SCORE_ALIBI = 1,
  ATTN_SCORE_SOFTCAP = 2,
  ATTN_SCORE_DROPOUT = 4   /* dropout on P (attn_fwd / attn_bwd, tensor-core path, d <= 128) */
};

/* Tile classes written by attn_classify_tiles. */
enum { ATTN_TILE_EMPTY = 0, ATTN_TILE_PARTIAL = 1, ATTN_TILE_FULL = 2 };

/* Side of the square tiles the kernels iterate over (query rows x key columns). */
#define ATTN_TILE 128

typedef struct {
  int32_t window;              /* ATTN_MASK_SLIDING_WINDOW: keys i-window+1 .. i */
  const int32_t* doc_offsets;  /* ATTN_MASK_DOCUMENT_CAUSAL: DEVICE int32[n_docs+1] */
  int32_t n_docs;
} attn_mask_params;

typedef struct {
  float softcap;               /* ATTN_SCORE_SOFTCAP: the cap c > 0 */
  float dropout_p;             /* ATTN_SCORE_DROPOUT: drop probability, 0 <= p < 1 */
  uint64_t dropout_seed;       /* ATTN_SCORE_DROPOUT: seed of the keep mask */
} attn_score_params;

/*
 * Dropout ("FlashAttention/es", "Variantes y sucesores": FlashAttention-1 supported
 * dropout). Element (i, j) of query head bh = b * Hq + h is kept iff byte j % 16 of
 * Philox4x32-10 (Salmon et al., SC 2011; 128-bit counter (j / 16, i, bh, 0), key = the
 * seed, low word first; byte k = bits 8 (k % 4) .. of word k / 4) is at least
 * floor(256 p) (capped at 255), so p is taken to 1/256; kept values are scaled by
 * 1 / (1 - p). The forward computes O = (P Z / (1 - p)) V with lse from the undropped
 * softmax; attn_bwd, given the same p and seed, regenerates Z: dV = (P Z / (1 - p))^T dO
 * and dS = P (dP Z / (1 - p) - D). Pass the same score_kind and score_params to both.
 */

/*
 * Forward pass ("FlashAttention/es", "El algoritmo FlashAttention"): writes
 * o = softmax(modified, masked scores) v and lse = m + log(l) per query row.
 * mask_params / score_params are HOST pointers and may be NULL when the kind
 * needs no parameter. Runs the tcgen05 tensor-core kernel.
 */
attn_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale,
                     int mask_kind, const attn_mask_params* mask_params,
                     int score_kind, const attn_score_params* score_params,
                     void* stream);

/*
 * Bytes of device workspace attn_bwd needs for these sizes (a multiple of 256): the
 * backward's per-query-row terms, computed by its first kernel. With
 * Nq128 = Nq rounded up to a multiple of 128 and R = B * Hq * Nq128, that is
 * 2 * round256(4 R) + round256(4 Nq128): L log2 e and D_i (one float each per padded
 * row) and each row's first allowed key (one int32 per padded row position).
 * 0 when B, Hq or Nq is 0.
 */
size_t attn_bwd_workspace_size(int B, int Hq, int Hkv, int Nq, int Nkv, int d);

/*
 * Backward pass ("FlashAttention/es", "Paso hacia atrás y recomputación"): from
 * q, k, v, the forward's o and lse, and the output gradient dout, rebuilds P
 * tile by tile and writes dq, dk, dv (bf16, overwritten, not accumulated). The
 * gradient algebra is the standard one: dV = P^T dO, dP = dO V^T,
 * D_i = rowsum(dO o O), dS = P o (dP - D) (times the soft-cap derivative),
 * dQ = scale dS K, dK = scale dS^T Q, with dK and dV summed over the query heads
 * of a group. workspace: DEVICE memory of at least attn_bwd_workspace_size bytes,
 * 256-byte aligned, not shared with a concurrent call.
 */
attn_status attn_bwd(const void* q, const void* k, const void* v, const void* o,
                     const float* lse, const void* dout, void* dq, void* dk, void* dv,
                     int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale,
                     int mask_kind, const attn_mask_params* mask_params,
                     int score_kind, const attn_score_params* score_params,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Kernels of the backward pass, for attn_bwd_phases. */
enum {
  ATTN_BWD_ROWDOT = 1,   /* row terms into the workspace: D = rowsum(dO o O), L log2 e,
                            first allowed key */
  ATTN_BWD_DKDV = 2,     /* dK and dV (reads the row terms) */
  ATTN_BWD_DQ = 4,       /* dQ (reads the row terms) */
  ATTN_BWD_ALL = 7
};

/*
 * attn_bwd split into its kernels: runs the ones named in `phases`, in the order
 * ROWDOT, DKDV, DQ, with attn_bwd's arguments and checks. DKDV and DQ read the row
 * terms from the workspace, so ROWDOT must have run on the same workspace and inputs before
 * them (in this call or an earlier one in stream order). DKDV and DQ do not depend
 * on each other: a caller may time them separately or put them on two streams.
 * attn_bwd(...) is attn_bwd_phases(ATTN_BWD_ALL, ...).
 */
attn_status attn_bwd_phases(int phases, const void* q, const void* k, const void* v,
                            const void* o, const float* lse, const void* dout, void* dq,
                            void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nkv, int d,
                            float scale, int mask_kind, const attn_mask_params* mask_params,
                            int score_kind, const attn_score_params* score_params,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass that allocates nothing and takes no workspace argument.
 *
 * The method on the pages has no counterpart of this call; it exists for callers
 * that cannot call cudaMalloc (or any allocator) where they run the backward pass:
 * for example a host program whose device memory is already handed out in full to
 * another allocator, or a runtime that forbids new allocations once it has started.
 * Such a caller still owns and passes every input and output, exactly as for
 * attn_bwd; only the backward's scratch (the per-query-row terms that
 * attn_bwd_workspace_size counts) lives in a fixed array inside this library instead
 * of a caller workspace.
 *
 * - The array holds 3 * ATTN_STATIC_WORKSPACE_ROWS 4-byte words (24 MiB) on every
 *   device that loads the library, for the life of the process. B * Hq * Nq128 (Nq
 *   rounded up to a multiple of 128) must not exceed ATTN_STATIC_WORKSPACE_ROWS;
 *   larger problems return ATTN_ERR_WORKSPACE and launch nothing (use attn_bwd with a
 *   workspace for them).
 * - The first call on a device looks up the array's device address with that device
 *   current (a one-time set-up per device); make that first call before any stream
 *   capture on the device.
 * - Every call on a device shares the one array, and the array keeps whatever the
 *   last call left there (each call overwrites every row it uses before reading it).
 *   Calls whose kernels can overlap on the GPU (other streams, other host threads)
 *   race on the array: order them on one stream or synchronise between them.
 * - Arguments, results, determinism and errors are otherwise those of attn_bwd.
 */
#define ATTN_STATIC_WORKSPACE_ROWS (1 << 21)
attn_status attn_bwd_static_workspace(const void* q, const void* k, const void* v,
                                      const void* o, const float* lse, const void* dout,
                                      void* dq, void* dk, void* dv, int B, int Hq, int Hkv,
                                      int Nq, int Nkv, int d, float scale, int mask_kind,
                                      const attn_mask_params* mask_params, int score_kind,
                                      const attn_score_params* score_params, void* stream);

/*
 * FP8 forward with block scales ("FlashAttention/es", "Variantes y sucesores", and
 * "FlashAttention-3 y torch.compile", section 2, name FP8 inputs for FlashAttention-3).
 * The inputs are e4m3 codes plus fp32 dequantisation scales, as written by
 * attn_quantize_fp8:
 *   q8   e4m3 [B, Hq, Nq, 128],  q_scale [B*Hq, ceil(Nq/128)]  (one per 128-row tile)
 *   k8   e4m3 [B, Hkv, Nkv, 128], k_scale [B*Hkv, ceil(Nkv/128)]
 *   v8t  e4m3 [B, Hkv, 128, attn_fp8_v_row_bytes(Nkv)] (V transposed, keys contiguous,
 *        zero padded), v_scale [B*Hkv] (one per head)
 * so that Q = q8 * q_scale etc. The result is attention (same masks and score mods as
 * attn_fwd) of those dequantised inputs, with P rounded to e4m3 (after a factor 2^7)
 * for the P V product: per element |O_ic - O_exact_ic| <= 2^-4 sum_j P_ij |V_jc|
 * + 2^-17 sum_j |V_jc| (over the row's allowed keys), plus bf16 rounding of O; lse is
 * exact up to fp32 rounding. d must be 128.
 * o: bf16 [B, Hq, Nq, 128]; lse: fp32 [B, Hq, Nq]. All pointers are DEVICE memory,
 * tensors 16-byte aligned, scales 4-byte aligned. Allocates nothing.
 */
attn_status attn_fwd_fp8(const void* q8, const void* k8, const void* v8t, const float* q_scale,
                         const float* k_scale, const float* v_scale, void* o, float* lse,
                         int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale,
                         int mask_kind, const attn_mask_params* mask_params, int score_kind,
                         const attn_score_params* score_params, void* stream);

/* Layouts of attn_quantize_fp8. */
enum {
  ATTN_FP8_TILES = 0,          /* Q, K: out [BH, N, d], scales [BH, ceil(N/128)] */
  ATTN_FP8_V_TRANSPOSED = 1    /* V: out [BH, d, attn_fp8_v_row_bytes(N)], scales [BH] */
};

/* Row length in bytes of the transposed e4m3 V: Nkv rounded up to 16 (0 if Nkv <= 0). */
size_t attn_fp8_v_row_bytes(int Nkv);

/*
 * bf16 x [BH, N, d] (d = 64 or 128, DEVICE) to e4m3 codes and fp32 scales: each
 * block (a 128-row tile for ATTN_FP8_TILES, a whole head for ATTN_FP8_V_TRANSPOSED)
 * gets s = amax / 448 (1 for an all-zero block) and code = e4m3(x / s), an IEEE fp32
 * division rounded to nearest even. Deterministic. x and out 16-byte aligned.
 */
attn_status attn_quantize_fp8(const void* x, void* out, float* scales, int BH, int N, int d,
                              int layout, void* stream);

/*
 * Decode over a paged KV cache ("FlashAttention/es", "Variantes y sucesores", names
 * PagedAttention, which cuts the inference KV cache into fixed-size pages shared by
 * many sequences). One call attends the Nq newest query tokens of each of B sequences
 * to every cached token of that sequence.
 *
 *   q          bf16 [B, Hq, Nq, d]  query i of sequence b sits at position
 *                                   seq_lens[b] - Nq + i (its own K/V are already in
 *                                   the cache)
 *   k_cache,   bf16 [num_pages, Hkv, page_size, d]: page p, kv head g, slot s
 *   v_cache
 *   page_table int32 [B, max_pages_per_seq]: token t of sequence b is in page
 *              page_table[b][t / page_size], slot t % page_size
 *   seq_lens   int32 [B]: cached tokens per sequence, 0 <= seq_lens[b] <= max_seq_len
 *   o          bf16 [B, Hq, Nq, d];  lse fp32 [B, Hq, Nq] (natural log)
 * All pointers are DEVICE memory; tensors 16-byte aligned, page_table and seq_lens
 * 4-byte aligned. page_table and seq_lens are read on the device only; a length
 * outside [0, max_seq_len] or a page index outside [0, num_pages) of a page that holds a
 * key of some query row makes attn_device_status report ATTN_ERR_DEVICE_INPUT (the results
 * of that call are then unspecified; nothing outside the given buffers is touched). Entries
 * of pages that a sliding window has passed for every query row may be anything.
 *
 * Masks use the positions above (aligned at the bottom right): ATTN_MASK_NONE (every
 * cached token), ATTN_MASK_CAUSAL (j <= position of the query), ATTN_MASK_SLIDING_WINDOW
 * (also position - j < window). ALiBi uses the signed distance position - j; soft-cap as
 * in attn_fwd. Document masking is not accepted (ATTN_ERR_ARG). Slots of a page past
 * the end of its sequence are never part of a result, whatever they hold.
 *
 * page_size: 8, 16, 32 or a multiple of 64. max_seq_len (<= max_pages_per_seq *
 * page_size) bounds seq_lens. split_keys (a positive multiple of 64, see
 * attn_decode_split_keys) cuts each sequence into chunks of that many keys, computed by
 * separate CTAs and merged by their log-sum-exp; with a single chunk
 * (max_seq_len <= split_keys) and more than 32 rows per query group no merge runs and no
 * workspace is needed. workspace:
 * DEVICE memory of attn_decode_workspace_size bytes, 256-byte aligned, not shared with
 * a concurrent call. Deterministic for fixed split_keys. Allocates nothing.
 */
attn_status attn_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* page_table, const int32_t* seq_lens, void* o,
                              float* lse, int B, int Hq, int Hkv, int Nq, int d, int num_pages,
                              int page_size, int max_pages_per_seq, int max_seq_len,
                              int split_keys, float scale, int mask_kind,
                              const attn_mask_params* mask_params, int score_kind,
                              const attn_score_params* score_params, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Workspace bytes of attn_decode_paged. The kernel keeps c copies of the rows of a kv
 * head's query group (G * Nq rows, G = Hq / Hkv) so that the softmax of a few rows is
 * spread over the SM: c = 2 for up to 32 rows, else 1. With
 * n = ceil(max_seq_len / split_keys) * c partial results per row and R = B * Hq * Nq
 * rows: round256(4 n R) + round256(4 n R d) (each partial's log2-sum-exp and normalised
 * fp32 output) when n > 1 and max_seq_len > 0, else 0.
 */
size_t attn_decode_workspace_size(int B, int Hq, int Hkv, int Nq, int d, int max_seq_len,
                                  int split_keys);

/*
 * A split_keys for attn_decode_paged: about ten work items (key chunks of one kv head
 * and 64-row query tile) per SM over total_kv_tokens (the sum of seq_lens, or
 * B * max_seq_len when unknown), a multiple of 64 and at least 256. Pure function of its
 * arguments.
 */
int attn_decode_split_keys(int B, int Hq, int Hkv, int Nq, long long total_kv_tokens,
                           int num_sms);

/*
 * ---- The paged cache as a whole: writing it, reading it back, attending chunks of new
 * tokens to it, and decode over an 8-bit cache ("FlashAttention/es", "Variantes y
 * sucesores": PagedAttention). One HOST struct describes a cache; its tensors are DEVICE
 * memory in attn_decode_paged's layout:
 *   k, v        [num_pages, Hkv, page_size, d]: page p, kv head g, slot s; bf16
 *               (ATTN_CACHE_BF16) or e4m3 codes, one byte each (ATTN_CACHE_E4M3)
 *   kv_exp      ATTN_CACHE_E4M3 only (NULL otherwise): uint8 [num_pages, Hkv, page_size, 2],
 *               the biased exponents of the K and of the V scale of each token and kv head:
 *               the value of a code is code * 2^(exp - 127)
 *   page_table  int32 [B, max_pages_per_seq], as in attn_decode_paged
 * d: 64 or 128; page_size: 8, 16, 32 or a multiple of 64; k, v, kv_exp 16-byte aligned.
 *
 * The calls take the packed rows of a ragged batch: offsets is int32 [B + 1] (DEVICE),
 * offsets[0] = 0, non-decreasing, offsets[B] <= T. Rows offsets[b] .. offsets[b+1] - 1 are
 * the n_b newest tokens of sequence b (n_b may be 0): row i of them sits at position
 * seq_lens[b] - n_b + i, where seq_lens int32 [B] (DEVICE) counts these tokens too. Rows of
 * a call behind offsets[B] belong to no sequence: they are neither read nor written.
 * Input rows may be strided views: element (t, h, c) of such a tensor is at
 * t * token_stride + h * head_stride + c (strides in elements, non-negative multiples of
 * 8; base 16-byte aligned), so the q, k and v slices of a fused projection need no copy.
 * Bad DEVICE inputs (offsets that break the rule above, a length above the page table's
 * capacity or max_seq_len, a page index outside [0, num_pages) of a page that the call reads
 * or writes, for cache_write and cache_read a position below 0) are skipped, never followed,
 * and reported by attn_device_status as ATTN_ERR_DEVICE_INPUT; the results of that call are
 * then unspecified. The calls allocate nothing, take any B and T (0 included) and are
 * deterministic.
 */
enum { ATTN_CACHE_BF16 = 0, ATTN_CACHE_E4M3 = 1 };

typedef struct {
  void* k;
  void* v;
  uint8_t* kv_exp;
  const int32_t* page_table;
  int32_t kind;                /* ATTN_CACHE_* */
  int32_t num_pages, Hkv, page_size, d;
  int32_t max_pages_per_seq;
} attn_paged_cache;

/*
 * Writes the K and V rows of the new tokens (bf16 [T, Hkv, d], strided) into the cache. A
 * bf16 cache takes them as they are. An e4m3 cache takes, per token and kv head and for K
 * and V apart, the smallest e with amax <= 448 * 2^e (amax: the largest finite magnitude of
 * the d values; e clamped to [-127, 127], -127 for a row of zeros), the codes
 * e4m3(x * 2^-e) rounded to nearest even, and the byte e + 127. A power-of-two scale costs
 * a floating-point code no precision, and code * 2^e is exact in bf16. NaN and infinities
 * become the NaN code. Slots of different new tokens must differ (two sequences may share
 * pages of older tokens, not the slot of a token that this call writes).
 */
attn_status attn_cache_write(const attn_paged_cache* cache, const void* k,
                             long long k_token_stride, long long k_head_stride, const void* v,
                             long long v_token_stride, long long v_head_stride,
                             const int32_t* offsets, const int32_t* seq_lens, int B, int T,
                             void* stream);

/*
 * Reads the newest tokens back: k, v bf16 [T, Hkv, d] (contiguous) receive the cached rows
 * (an e4m3 cache: code * 2^e, rounded to bf16, which is exact for what attn_cache_write
 * wrote down to bf16's smallest normal value). With n_b = seq_lens[b] this is the whole
 * sequence.
 */
attn_status attn_cache_read(const attn_paged_cache* cache, void* k, void* v,
                            const int32_t* offsets, const int32_t* seq_lens, int B, int T,
                            void* stream);

/*
 * Attention of a ragged batch of chunks of new tokens over the cache (chunked prefill; the
 * new tokens' own K and V are in the cache already, see attn_cache_write).
 *   q    bf16 [T, Hq, d], strided;  o bf16 [T, Hq, d];  lse fp32 [T, Hq] (natural log)
 * Masks, ALiBi, soft-cap and their positions are those of attn_decode_paged. Of a sliding
 * window's sequence only the pages that hold a key of some query row are read
 * (attn_decode_paged_e4m3 too): the entries of the pages below may be anything. A row without
 * an allowed key gets O = 0 and lse = -inf. max_new bounds every n_b and max_seq_len
 * (<= max_pages_per_seq * page_size) every seq_lens[b]; tighter bounds launch fewer CTAs.
 * split_keys (a positive multiple of 128, see attn_prefill_split_keys) cuts the keys into
 * chunks computed by separate CTAs and merged by their log-sum-exp; with
 * max_seq_len <= split_keys no merge runs and no workspace is needed. workspace: DEVICE
 * memory of attn_prefill_workspace_size bytes, 256-byte aligned, not shared with a
 * concurrent call (two captured graphs that may run at the same time need one each).
 * An e4m3 cache is attended to as the values its codes stand for: exactly while the K scales,
 * and the V scales, of the keys that a query's tile walks over lie within 2^15 of each
 * other, and within bf16's rounding up to 2^24 (attn_decode_paged_e4m3 too). Over such a cache
 * the softmax weights that multiply V are rounded to 11 bits, those below 2^-17 of the row's
 * largest to multiples of 2^-27 of it; the row sum is not. Over a bf16 cache O is summed
 * before it is divided by the row sum (attn_decode_paged too): it needs max |V| times the keys
 * that share the weight below 2^119. A NaN in a query
 * row, or in the K row of a token that it sees, makes that row's O and lse NaN and no
 * other's. A NaN or infinity in the V row of a cached token reaches O in every query row of
 * the tiles that hold the token, those that mask it too (0 * NaN).
 */
attn_status attn_prefill_paged(const attn_paged_cache* cache, const void* q,
                               long long q_token_stride, long long q_head_stride, void* o,
                               float* lse, const int32_t* offsets, const int32_t* seq_lens,
                               int B, int T, int Hq, int max_new, int max_seq_len,
                               int split_keys, float scale, int mask_kind,
                               const attn_mask_params* mask_params, int score_kind,
                               const attn_score_params* score_params, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Workspace bytes of attn_prefill_paged: with n = ceil(max_seq_len / split_keys) and
 * R = T * Hq rows, round256(4 n R) + round256(4 n R d) when n > 1, else 0.
 */
size_t attn_prefill_workspace_size(int T, int Hq, int d, int max_seq_len, int split_keys);

/*
 * A split_keys for attn_prefill_paged over a cache of this kind (ATTN_CACHE_*): all keys in
 * one chunk when the row tiles alone fill the SMs, else chunks of at least 1024 keys,
 * several per SM over total_kv_tokens (the sum of seq_lens, or B * max_seq_len when
 * unknown). attn_decode_paged_e4m3 takes its result too (T = B * Nq, max_new = Nq). Pure
 * function of its arguments.
 */
int attn_prefill_split_keys(int cache_kind, int B, int T, int Hq, int Hkv, int max_new,
                            int max_seq_len, long long total_kv_tokens, int num_sms);

/*
 * attn_decode_paged over an ATTN_CACHE_E4M3 cache: same queries, outputs, masks, score
 * modifications and split_keys. The workspace holds one partial result per chunk and row:
 * attn_prefill_workspace_size(B * Nq, Hq, d, max_seq_len, split_keys) bytes.
 */
attn_status attn_decode_paged_e4m3(const attn_paged_cache* cache, const void* q,
                                   const int32_t* seq_lens, void* o, float* lse, int B, int Hq,
                                   int Nq, int max_seq_len, int split_keys, float scale,
                                   int mask_kind, const attn_mask_params* mask_params,
                                   int score_kind, const attn_score_params* score_params,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * ---- Who holds which page: the cache's pages forked, grown, rolled back, given back,
 * compacted and copied on the device, so that a serving loop needs no host round trip
 * ("FlashAttention/es", "Variantes y sucesores": PagedAttention's pages are shared by many
 * sequences). Three int32 DEVICE tensors hold the state, changed in place by these calls:
 *   page_table  [B, max_pages_per_seq]: as in attn_decode_paged. Row b holds the pages of
 *               entries 0 .. ceil(seq_lens[b] / page_size) - 1; a negative entry among them
 *               holds none (a sliding window has passed it). Entries behind are not read.
 *   seq_lens    [B]
 *   page_refs   [num_pages]: how many table entries hold the page, plus whatever else the
 *               caller counts as a holder (a prefix kept for later); a page with 0 is free
 * The tensors of one call must not overlap. Bad DEVICE inputs (a length outside [0,
 * max_pages_per_seq * page_size], an entry at or above num_pages that the call reads, a parent
 * at or above B) are skipped, never followed, and reported by attn_device_status as
 * ATTN_ERR_DEVICE_INPUT; the results of that call are then unspecified. A roll-back into a page
 * that the table has given up (a window's) is such an input for the call that grows the row
 * again. The calls allocate nothing, take any B (0
 * included, attn_cache_fork up to 49152) and are deterministic. workspace: DEVICE memory of
 * the size that the call's size function gives, 256-byte aligned, not shared with a concurrent
 * call (two captured graphs that may run at the same time need one each).
 */

/*
 * Row i takes over what row parents[i] (int32 [B]) held before the call: its entries and its
 * length; a negative parent leaves row i empty, parents[i] = i leaves it as it is. Several rows
 * may have one parent (beams, samples of one prompt) and share its pages then, the last,
 * partly filled one too: attn_cache_resize copies that page before one of them writes into
 * it. Pages lose the holders that let go of them; those of no holder are free. Entries that
 * no longer hold a page of their row become -1.
 */
attn_status attn_cache_fork(int32_t* page_table, int32_t* seq_lens, int32_t* page_refs,
                            const int32_t* parents, int B, int max_pages_per_seq, int num_pages,
                            int page_size, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of attn_cache_fork: round256(4 B max_pages_per_seq) + 2 round256(4 B). */
size_t attn_fork_workspace_size(int B, int max_pages_per_seq);

/*
 * Takes every row from seq_lens[b] to new_lens[b] tokens (int32 [B]): room for new tokens
 * before attn_cache_write, a roll-back of drafted tokens that were not accepted, or 0 for a
 * sequence that has ended. In this order:
 *   1. Rows give back the entries behind their new length and, with window > 0, the pages
 *      wholly below position min(seq_lens[b], new_lens[b]) - window + 1, the lowest one that a
 *      sliding window leaves visible to the tokens to come: from there down to the next entry
 *      that holds no page. Their entries become -1.
 *   2. A row that grows from inside a page writes into that page. Where others hold it too the
 *      row takes a new page and the tokens that it has there are copied (K, V and scales): of
 *      the g rows that write into a page with r holders all do if r > g, else all but the
 *      lowest row.
 *   3. Rows take the pages for their new tokens. Free pages (those given back in step 1 are
 *      among them) are handed out in ascending order, rows in order, a row's copied page first.
 * If the pages do not suffice nothing is changed, and *missing (DEVICE int32) says how many
 * lack; else it is 0. seq_lens do not count the new tokens then: attn_cache_write,
 * attn_prefill_paged and attn_verify_drafts would take the last cached tokens for the rows of the
 * chunk, the first overwriting them, in shared pages too. A caller that goes on without reading
 * *missing gives those calls offsets that are all zero if *missing is not 0 (offsets times
 * (*missing == 0)): no rows, nothing written, kept_lens equal to seq_lens.
 * Only the cache's sizes, kind, k, v and kv_exp are used (cache->page_table
 * is not read). What new pages hold behind the copied tokens stays.
 */
attn_status attn_cache_resize(const attn_paged_cache* cache, int32_t* page_table,
                              int32_t* seq_lens, int32_t* page_refs, const int32_t* new_lens,
                              int B, int window, int32_t* missing, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Workspace bytes of attn_cache_resize: 6 round256(4 B) + 2 round256(4 num_pages) +
 * round256(4 min(num_pages, B max_pages_per_seq)) + 256.
 */
size_t attn_resize_workspace_size(int B, int max_pages_per_seq, int num_pages);

/*
 * Moves the used pages (page_refs != 0) to the front of the pool: with U of them, the k-th
 * highest used page at or above U moves to the k-th lowest free page below it, with its count,
 * and the table's entries follow (held ones alone). Afterwards pages U .. num_pages - 1 are free:
 * the pool can be cut there. *used (DEVICE int32) receives U and page_map (DEVICE int32
 * [num_pages]) each page's new index, -1 for a free page, for holders outside of the table.
 * Only the cache's sizes, kind, k, v and kv_exp are used (cache->page_table is not read).
 */
attn_status attn_cache_compact(const attn_paged_cache* cache, int32_t* page_table,
                               const int32_t* seq_lens, int32_t* page_refs, int B, int32_t* used,
                               int32_t* page_map, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Workspace bytes of attn_cache_compact: 2 round256(4 num_pages) + 256. */
size_t attn_compact_workspace_size(int num_pages);

/*
 * Copies page src_pages[i] of one pool to page dst_pages[i] of another (int32 [n]), K, V and
 * scales, for i = 0 .. n - 1: to another engine's pool, or out of the way and back. Both caches
 * agree in kind, Hkv, page_size and d; their page tables are not read. An entry with a negative
 * page is skipped. `to` may be the same pool as `from`, described with other num_pages too (pools
 * without bytes count as two); pools that overlap in any other way are refused (ATTN_ERR_ARG). Every source is read as it was before the call: of the entries with one
 * destination only the first is copied, and within one pool none whose source is another entry's
 * destination (an entry that copies a page to itself is good, if it is the first with that
 * destination); the entries left out, and pages outside the pools, are reported
 * (ATTN_ERR_DEVICE_INPUT) while the others are copied. Counts and tables are the caller's.
 */
attn_status attn_cache_copy(const attn_paged_cache* from, const attn_paged_cache* to,
                            const int32_t* src_pages, const int32_t* dst_pages, int n,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of attn_cache_copy: round256(4 num_pages of `to`), whatever n. */
size_t attn_copy_workspace_size(int num_pages_to, int n);

/* Types of probabilities. */
enum { ATTN_PROB_FP32 = 0, ATTN_PROB_BF16 = 1, ATTN_PROB_FP16 = 2 };

/*
 * Verification of drafted tokens (speculative decoding), after attn_prefill_paged has scored
 * them: decides from given random numbers which of a sequence's drafts stay, and draws the
 * token that follows, so that the tokens are distributed as the target's own.
 *
 * The call takes the packed rows of the scored chunks: offsets int32 [B + 1] as in
 * attn_prefill_paged. Row 0 of a sequence's n rows is the token it ended in, rows 1 .. n - 1 are
 * its drafts (tokens int32 [T]; row 0's is not read).
 *   target  [T, V] probabilities of the token after each row
 *   draft   [T, V], row t: the probabilities that tokens[t + 1] was drawn from (the last row of
 *           a sequence is not read); NULL for drafts that were not drawn (looked up): they count
 *           as drawn from a distribution that has all its weight on them
 *           both of prob_type, element (t, x) at t * stride + x (any stride in elements)
 *   accept_u fp32 [T], sample_u fp32 [B]: random numbers, uniform in [0, 1)
 * Draft x of row t stays iff accept_u[t] * draft[t, x] < target[t, x] (exactly, without
 * rounding) and the drafts before it stay. accepted[b] (int32 [B]) of them stay. If that is all
 * n - 1, the next token is drawn from the last row of target, else from
 * max(target[t] - draft[t], 0) of the first row t whose draft does not stay (from target[t] if
 * that is zero everywhere): next_tokens[b] (int32 [B]) is the lowest x whose cumulative weight
 * exceeds sample_u[b] times the total weight (the last with any weight if rounding leaves
 * none). Rows need not sum to one; what is not a positive finite number has no weight, and a
 * draft without a positive finite target probability or a finite draft probability does not stay.
 * Sums are held as pairs of fp32 numbers: where sample_u[b] times the total lies closer than 2^-32 of
 * the total to the border between two tokens (V up to 2^20) the token may be either. A sequence
 * without rows gets 0 and -1; one whose row has no weight, or weights that sum to more than fp32 holds,
 * gets -1 and is reported (ATTN_ERR_DEVICE_INPUT), as are offsets that break the rule and a draft
 * outside [0, V), which does not stay.
 * With seq_lens (int32 [B], the cached tokens with all rows of the chunk; else NULL)
 * kept_lens[b] = seq_lens[b] - (drafts that do not stay): attn_cache_resize takes it.
 * The outputs are DEVICE tensors. Allocates nothing; deterministic.
 */
attn_status attn_verify_drafts(int prob_type, const void* target, long long target_stride,
                               const void* draft, long long draft_stride, const int32_t* tokens,
                               const int32_t* offsets, const float* accept_u,
                               const float* sample_u, const int32_t* seq_lens, int B, int T, int V,
                               int32_t* accepted, int32_t* next_tokens, int32_t* kept_lens,
                               void* stream);

/*
 * Block-sparsity classifier ("El FlexAttention de PyTorch con FlashAttention-4 es
 * un cambio radical", "Limitaciones actuales", names block sparsity): writes
 * classes[r * ceil(Nkv/128) + c] = EMPTY / PARTIAL / FULL for query tile r and key
 * tile c, with the same tile rule the forward and backward kernels use to skip
 * and to mask tiles. classes: DEVICE int32 [ceil(Nq/128) * ceil(Nkv/128)].
 */
attn_status attn_classify_tiles(int mask_kind, const attn_mask_params* mask_params,
                                int Nq, int Nkv, int32_t* classes, void* stream);

/*
 * Checks a document-offsets table on the device: doc_offsets[0] = 0, non-decreasing,
 * doc_offsets[n_docs] = N (the contract of ATTN_MASK_DOCUMENT_CAUSAL). A violation is
 * not returned here (the table is device memory and the call is asynchronous): it is
 * recorded in the device status word, which the next attn_device_status reports as
 * ATTN_ERR_DEVICE_INPUT. Reads doc_offsets[0 .. n_docs] only (DEVICE int32, 4-byte
 * aligned). Returns ATTN_ERR_ARG for a null pointer, n_docs < 1 or N < 0.
 *
 * Checked mode: when the environment variable ATTN_CHECKED holds a value other than
 * "" or "0" at the library's first look at it (once per process), every call with
 * ATTN_MASK_DOCUMENT_CAUSAL (attn_fwd, attn_bwd and their variants, attn_fwd_fp8,
 * attn_classify_tiles) first runs this check on its table, in stream order before its
 * own kernels. The kernels of a call still run on a bad table; they read and write
 * only inside their buffers whatever the offsets hold, but their results are then
 * meaningless. The mode is for debugging; by default the table is trusted.
 */
attn_status attn_check_doc_offsets(const int32_t* doc_offsets, int n_docs, int N,
                                   void* stream);

/*
 * Plain CUDA-core versions of the forward and backward passes (one thread per
 * row, fp32 arithmetic, no tensor cores). They exist to cross-check the tensor-core
 * kernels and are never chosen automatically. Same arguments and contract as
 * attn_fwd / attn_bwd (attn_bwd_simt needs the same workspace).
 */
attn_status attn_fwd_simt(const void* q, const void* k, const void* v, void* o, float* lse,
                          int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale,
                          int mask_kind, const attn_mask_params* mask_params,
                          int score_kind, const attn_score_params* score_params,
                          void* stream);
attn_status attn_bwd_simt(const void* q, const void* k, const void* v, const void* o,
                          const float* lse, const void* dout, void* dq, void* dk, void* dv,
                          int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale,
                          int mask_kind, const attn_mask_params* mask_params,
                          int score_kind, const attn_score_params* score_params,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Self-test of the failure path every kernel shares: launches one warp whose wait on a
 * shared-memory barrier that nothing completes is the library's bounded wait. After the
 * wait limit (2 s of the device clock) it gives up and records ATTN_ERR_DEVICE_TIMEOUT
 * in the device status word, which attn_device_status then reports and clears; the
 * context stays usable. Asynchronous on `stream`. Returns ATTN_ERR_ARCH or
 * ATTN_ERR_LAUNCH if the kernel cannot be launched.
 */
attn_status attn_selftest_wait_timeout(void* stream);

/*
 * Synchronises `stream` and reports whether a kernel of this library on the
 * current device gave up a bounded wait since the last call (ATTN_ERR_DEVICE_TIMEOUT),
 * met an out-of-range device input (ATTN_ERR_DEVICE_INPUT), or whether the stream
 * itself failed (ATTN_ERR_LAUNCH). Clears the flags.
 */
attn_status attn_device_status(void* stream);

/* Static, human-readable text for a status code. */
const char* attn_strerror(attn_status status);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_IO_AWARE_ATTN_H */
