// Copies of cache pages that a plan kernel has listed (pool.cu): the partial pages that a resize
// copies before they are written, the pages that a compaction moves, and pages copied between
// pools. A whole page is one run of Hkv * page_size rows per tensor, the first tokens of a page
// one run per kv head. Bound by HBM: every byte is read once and written once.
#include "paged.cuh"
#include "pool.cuh"

namespace attn {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kChunk = 16384;  // bytes of one run that a CTA copies at a time

// Table entries of the rows after a compaction.
__device__ void rewrite_table(const CompactArgs& c) {
  const PoolState& s = c.s;
  const int lane = threadIdx.x & 31;
  const int U = __ldcg(c.used);
  const int warps = gridDim.x * (kCopyThreads / 32);
  for (int b = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); b < s.B; b += warps) {
    const int L = __ldg(s.lens + b);
    if (!length_ok(s, L)) {
      atomicOr(s.status, DEV_BAD_INPUT);
      continue;
    }
    int32_t* row = s.table + (size_t)b * s.max_pages;
    for (int i = lane, n = pages_of(s, L); i < n; i += 32) {
      const int page = row[i];
      if (page < U) continue;  // not moved, or no page
      const int to = page < s.num_pages ? __ldcg(c.page_map + page) : -1;
      if (to < 0) atomicOr(s.status, DEV_BAD_INPUT);
      else row[i] = to;
    }
  }
}

// Copies n bytes (a multiple of 2; both addresses 16-byte aligned) with the CTA's threads.
__device__ __forceinline__ void copy_run(const uint8_t* from, uint8_t* to, int n) {
  for (int i = threadIdx.x * 16; i + 16 <= n; i += kCopyThreads * 16)
    *reinterpret_cast<uint4*>(to + i) = __ldg(reinterpret_cast<const uint4*>(from + i));
  const int tail = (n & ~15) + (int)threadIdx.x * 2;
  if (tail < n) *reinterpret_cast<uint16_t*>(to + tail) = __ldg(reinterpret_cast<const uint16_t*>(from + tail));
}

template <bool kCompact>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageCopy c, const CompactArgs compact) {
  grid_dependency_wait();
  if constexpr (kCompact) rewrite_table(compact);
  const int count = __ldcg(c.moves.count);
  if (count == 0) return;
  const int heads = c.moves.tokens ? c.Hkv : 1;
  const int row_bytes = c.e4m3 ? c.d : 2 * c.d;
  const long long run = (long long)(c.moves.tokens ? 1 : c.Hkv) * c.page_size;  // tokens of a run
  const long long page_rows = (long long)c.Hkv * c.page_size;
  const int chunks = (int)((run * row_bytes + kChunk - 1) / kChunk);
  const int exp_chunks = c.e4m3 ? (int)((run * 2 + kChunk - 1) / kChunk) : 0;
  const int per_head = 2 * chunks + exp_chunks;
  const long long per_move = (long long)heads * per_head, units = count * per_move;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int move = (int)(u / per_move), rest = (int)(u - move * per_move);
    const int src = __ldcg(c.moves.src + move);
    if (src < 0) continue;
    const int dst = __ldcg(c.moves.dst + move);
    const int head = rest / per_head, part = rest - head * per_head;
    const int which = part < chunks ? 0 : part < 2 * chunks ? 1 : 2;
    const long long at = (long long)(part - which * chunks) * kChunk;
    const int bytes = which == 2 ? 2 : row_bytes;
    const long long n = (c.moves.tokens ? (long long)__ldcg(c.moves.tokens + move) : run) * bytes - at;
    if (n <= 0) continue;
    const long long off = (long long)head * c.page_size * bytes + at, page = page_rows * bytes;
    copy_run(static_cast<const uint8_t*>(c.from[which]) + src * page + off,
             static_cast<uint8_t*>(c.to[which]) + dst * page + off, (int)imin64(n, kChunk));
  }
}

}  // namespace

cudaError_t launch_page_copy(const PageCopy& c, const CompactArgs* compact, int num_sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((num_sms > 0 ? num_sms : 1) * 8);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return compact ? cudaLaunchKernelEx(&cfg, page_copy_kernel<true>, c, *compact)
                 : cudaLaunchKernelEx(&cfg, page_copy_kernel<false>, c, CompactArgs{});
}

}  // namespace attn
