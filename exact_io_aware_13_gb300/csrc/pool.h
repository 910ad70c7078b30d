// Host-side launch interface of the kernels around the paged cache: which sequence holds which
// page (fork, resize, compact), page copies, and the verification of drafted tokens.
#pragma once

#include "attn.h"
#include "paged.h"
#include "pool_rules.h"

namespace attn {

// The integers that say who holds which page (include/attn.h). All device memory.
struct PoolState {
  int32_t* table;   // [B, max_pages]
  int32_t* lens;    // [B]
  int32_t* refs;    // [num_pages]
  int* status;
  int B, max_pages, num_pages;
  int page_size, page_shift;  // page_shift: log2 page_size, or -1
};

// Copies of pages that a plan kernel has listed: entry i < *count takes tokens 0 .. tokens[i] - 1
// (without `tokens` the whole page) of page src[i] to page dst[i]; a negative src is no copy.
// The copies of a list touch disjoint bytes.
struct PageMoves {
  int32_t* count;
  int32_t *src, *dst, *tokens;
  int most;  // bound on *count
};
struct PageCopy {
  const void* from[3];  // K, V codes or values [pages, Hkv, page_size, d], kv_exp or null
  void* to[3];
  int Hkv, page_size, d;
  bool e4m3;
  int* status;
  PageMoves moves;
  int runs, kv_pieces, exp_pieces;  // of a move; set by the launch
};

struct ForkArgs {
  PoolState s;
  const int32_t* parents;  // [B]
  int32_t* rows;           // workspace [B, max_pages]: the new rows
  int32_t *old_lens, *new_lens;  // workspace [B] each
};
struct ResizeArgs {
  PoolState s;
  const int32_t* new_lens;  // [B]
  int window;
  int32_t* missing;
  int32_t *write_page, *row_rank, *row_move;  // workspace [B] each
  int32_t *writers, *lowest;                  // workspace [num_pages] each
  int32_t* free_list;                         // workspace [min(num_pages, B * max_pages)]
  PageMoves moves;                            // [B]
};
struct CompactArgs {
  PoolState s;
  int32_t *used, *page_map;
  PageMoves moves;  // [num_pages]
};
constexpr int kMaxCopyEntries = 1 << 30;  // of a caller's list
// A caller's list of page copies. Of the entries with one destination the first is copied; within
// one pool an entry whose source is another's destination is not.
struct CopyList {
  const int32_t *src, *dst;  // [n]
  int n, num_pages_from, num_pages_to;
  bool same_pool;
  int32_t* owner;  // workspace [num_pages_to]: the first entry with that destination
  int* status;
};
// Whether clusters of kPlanMaxCtas, the only size above the portable one in use, can run this
// kernel with cfg's block and shared memory: asked once per device. known, yes: one bit per device,
// statics of the launch site's kernel.
bool large_clusters(const void* kernel, const cudaLaunchConfig_t& cfg, std::atomic<uint64_t>& known,
                    std::atomic<uint64_t>& yes);

// Rows of one fork: their counters fill a CTA's shared memory.
constexpr int kForkMaxRows = 49152;
cudaError_t launch_fork(const ForkArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_resize(const ResizeArgs& a, const PageCopy& c, int num_sms, cudaStream_t st);
cudaError_t launch_compact(const CompactArgs& a, const PageCopy& c, int num_sms, cudaStream_t st);
cudaError_t launch_copy_pages(const CopyList& l, const PageCopy& c, int num_sms, cudaStream_t st);
// The copies of a plan, behind the kernel that lists them; a compaction's table entries are
// rewritten in the same launch.
cudaError_t launch_page_copy(const PageCopy& c, int num_sms, cudaStream_t st);
cudaError_t launch_compact_copy(const PageCopy& c, const CompactArgs& compact, int num_sms, cudaStream_t st);

// Verification of drafted tokens.
struct VerifyArgs {
  const void *target, *draft;             // [T, V] rows, draft may be null
  long long target_stride, draft_stride;  // elements
  const int32_t* tokens;                  // [T]
  const int32_t* offsets;                 // [B + 1]
  const float *accept_u, *sample_u;       // [T], [B]
  const int32_t* seq_lens;                // [B] or null
  int32_t *accepted, *next_tokens, *kept_lens;  // [B]; kept_lens null without seq_lens
  int* status;
  int B, T, V;
  int type;                               // ATTN_PROB_*
};
constexpr int kVerifyMaxRows = 1 << 26;  // sequences of a call: clusters of a grid
constexpr int kVerifyMaxTokens = 1 << 30;  // of a vocabulary
cudaError_t launch_verify(const VerifyArgs& a, int num_sms, cudaStream_t st);

}  // namespace attn
