// Host-side launch interface of the paged cache's kernels (the rest is in kernels.h).
#pragma once

#include <atomic>

#include "kernels.h"

namespace attn {

// Raises a kernel's dynamic shared-memory limit, once per kernel and device (the call costs a
// launch about 1 us). `done`: one bit per device, a static of the launch site.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- Paged cache: write, read back, chunk attention, e4m3 decode.
// A cache and a ragged batch of packed rows over it (include/attn.h). Row (t, h) of a
// strided [T, H, d] tensor starts at element t * token_stride + h * head_stride. Decode has
// no offsets: sequence b's rows are b * max_new .. b * max_new + max_new - 1.
struct PagedProblem {
  void *k_cache, *v_cache;    // [num_pages, Hkv, page_size, d], bf16 or e4m3
  uint8_t* kv_exp;            // [num_pages, Hkv, page_size, 2] (e4m3)
  const int32_t* page_table;  // [B, max_pages] device
  const int32_t* offsets;     // [B + 1] device, or null
  const int32_t* seq_lens;    // [B] device
  int* status;
  bool e4m3;                  // codes and kv_exp, else bf16
  int num_pages, Hkv, page_size, d, max_pages;
  int page_shift;             // log2 page_size, or -1
  int B, T;
  int max_new;                // bound on the new tokens of a sequence
  int max_seq_len;            // bound on seq_lens (<= max_pages * page_size)
};
struct RowView {
  const __nv_bfloat16* p;
  long long token_stride, head_stride;
};
cudaError_t launch_cache_write(const PagedProblem& p, const RowView& k, const RowView& v,
                               cudaStream_t st);
cudaError_t launch_cache_read(const PagedProblem& p, __nv_bfloat16* k, __nv_bfloat16* v,
                              cudaStream_t st);

// Attention over the cache.
struct PagedAttention {
  PagedProblem p;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  // element offsets of row (b, i, h): b * batch + t * token + h * head, with t the packed
  // row (chunks; batch = 0) or the query index i (decode)
  long long q_batch, q_token, q_head;
  long long o_batch, o_token, o_head;
  long long l_batch, l_token, l_head;
  int Hq, G;                  // query heads; query heads per kv head
  float scale, softcap;
  int score_kind, mask_kind, window;
  int chunk, n_chunks;        // keys per split (n_chunks = 1: one chunk holds every key)
  float* part_o;              // [n_chunks, T * Hq, d] fp32 when n_chunks > 1
  float* part_lse;            // [n_chunks, T * Hq]
};
// Tensor maps over the cache's rows. Row kernel (e4m3): whole rows of d codes, boxes of
// min(page_size, 32) rows, swizzled over the row. Tile kernel, bf16: boxes of 64 columns and
// min(page_size, 64) rows, 128-byte swizzle (e4m3 tiles come by bulk copies, without a map).
struct PagedMaps {
  CUtensorMap k, v;
};
// Few query rows per kv head over an e4m3 cache take the row kernel: 32 rows over 16 long
// caches ran in 233 us there, in 339 us as tiles (both with a merge 9 us slower than now); with
// 64 rows it would read every key twice.
constexpr int kPagedRowsMax = 32;
inline bool paged_few_rows(const PagedAttention& a) {
  return a.p.e4m3 && (long long)a.p.max_new * a.G <= kPagedRowsMax;
}
cudaError_t launch_paged_rows(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st);
cudaError_t launch_paged_tiles_bf16(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st);
cudaError_t launch_paged_tiles_e4m3(const PagedAttention& a, cudaStream_t st);
cudaError_t launch_paged_attention(const PagedAttention& a, const PagedMaps& maps,
                                   cudaStream_t st);

}  // namespace attn
