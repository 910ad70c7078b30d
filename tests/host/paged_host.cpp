// Host-only build of the paged cache's index rules (csrc/paged_index.cuh) so that the tests
// can run them on the CPU against bad offsets, lengths and page indices.
#include "paged_index.cuh"

extern "C" {

int host_span_ok(int T, int max_new, int max_seq_len, int o0, int o1, int L) {
  return attn::paged_span_ok(T, max_new, max_seq_len, o0, o1, L) ? 1 : 0;
}

long long host_row(int page, int num_pages, int Hkv, int page_size, int head, int slot) {
  return attn::paged_row(page, num_pages, Hkv, page_size, head, slot);
}

int host_skipped_keys(int t0, int k_lo, int R) { return attn::paged_skipped_keys(t0, k_lo, R); }

// (page, slot) of key0, key0 + stride, ... (n of them), by the walk.
void host_walk(int key0, int stride, int page_size, int n, int* pages, int* slots) {
  attn::PageWalk w(key0, page_size);
  for (int i = 0; i < n; ++i) {
    pages[i] = w.page;
    slots[i] = w.slot;
    w.advance(stride, page_size);
  }
}

}  // extern "C"
