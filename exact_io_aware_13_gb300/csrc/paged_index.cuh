// Index arithmetic of the paged cache that follows device inputs: what is checked before an
// offset, a length or a page index is used. Compiles on the host too, where the tests run it
// against bad inputs.
#pragma once

#include <cstdint>

#include "mask.cuh"

namespace attn {

ATTN_HD long long imin64(long long a, long long b) { return a < b ? a : b; }

// Whether a sequence's packed rows [o0, o1) and length can be used: inside the call's T rows
// and bounds.
ATTN_HD bool paged_span_ok(int T, int max_new, int max_seq_len, int o0, int o1, int L) {
  return o0 >= 0 && o1 >= o0 && o1 <= T && o1 - o0 <= max_new && L >= 0 && L <= max_seq_len;
}

// Row (page * Hkv + head) * page_size + slot of the cache's [num_pages * Hkv * page_size, d]
// rows, or -1 for a page outside the pool.
ATTN_HD long long paged_row(int page, int num_pages, int Hkv, int page_size, int head, int slot) {
  if (page < 0 || page >= num_pages) return -1;
  return ((long long)page * Hkv + head) * page_size + slot;
}

// Keys at the start of the tile at t0 that are not loaded: the page pieces of R keys (a power of
// two) that end at or below k_lo, the lowest key that any row of the CTA sees. Their pages may be gone (a sliding
// window has passed them) or be another sequence's by now; their V rows count as zeros.
ATTN_HD int paged_skipped_keys(int t0, int k_lo, int R) {
  return k_lo > t0 ? (k_lo - t0) & -R : 0;
}

// The page-table index and slot of a key that moves on by a fixed stride (a power of two,
// 64 or 128), without a division: a page size of at most the stride divides it (8, 16, 32,
// 64, 128), so the slot stays; a larger one is passed at most once.
struct PageWalk {
  int page, slot;
  ATTN_HD PageWalk(int key, int page_size) : page(key / page_size), slot(key % page_size) {}
  ATTN_HD void advance(int stride, int page_size) {
    if (page_size <= stride) {
      page += stride / page_size;
    } else if ((slot += stride) >= page_size) {
      slot -= page_size;
      ++page;
    }
  }
};

}  // namespace attn
