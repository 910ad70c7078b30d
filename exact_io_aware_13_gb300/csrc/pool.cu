// Plans of the pool's operators: who holds which page after a fork, a resize or a compaction,
// and which pages have to be copied for it (pool_copy.cu copies them).
//
// Everything here is integer work with one answer: free pages are handed out in ascending
// order, rows take them in order, and counters are sums, so no order of atomics shows. Each
// plan reads the counts of all pages at most twice (4 bytes a page) and the table entries that
// change; it is bound by the latency of its few steps, not by bytes: 512 beams of up to 1024 pages
// forked in 9 us, 64 rows over 4900 pages grown by a token in 8 us (the copy kernel behind it, 1 us
// where there is nothing to copy, not counted), 160 rows over 99500 pages with a window in 17 us, 8660 pages
// planned for compaction in 6 us.
#include "paged.cuh"
#include "pool.cuh"

namespace attn {

bool large_clusters(const void* kernel, const cudaLaunchConfig_t& cfg, std::atomic<uint64_t>& known,
                    std::atomic<uint64_t>& yes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  const uint64_t bit = 1ull << dev;
  if (known.load(std::memory_order_acquire) & bit) return yes.load(std::memory_order_acquire) & bit;
  // (the answer is kept, so the question is one of sizes that do not change from call to call)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanMaxCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t ask = cfg;
  ask.gridDim = dim3(kPlanMaxCtas);
  ask.attrs = attr;
  ask.numAttrs = 1;
  int clusters = 0;
  const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&clusters, kernel, &ask) == cudaSuccess && clusters > 0;
  if (!ok) cudaGetLastError();
  if (ok) yes.fetch_or(bit, std::memory_order_release);
  known.fetch_or(bit, std::memory_order_release);
  return ok;
}

namespace {

__device__ __forceinline__ void report(const PoolState& s) { atomicOr(s.status, DEV_BAD_INPUT); }

// Adds n to the holders of a table entry's page; an entry behind the pool is reported.
__device__ __forceinline__ void add_refs(const PoolState& s, int page, int n) {
  if (page < 0) return;
  if (page >= s.num_pages) report(s);
  else atomicAdd(s.refs + page, n);
}

// ---------------------------------------------------------------- fork
// Row i takes what row parents[i] held. A row r that c rows take adds c - 1 holders to each of
// its pages. The new rows are gathered into the workspace before any row is overwritten: in one
// cluster (kBoth) for few entries, else in two launches over all SMs. A warp takes kForkChunk
// entries of a row at a time, a lane's loads all in flight.
enum ForkPhase { kGather = 1, kScatter = 2, kBoth = 3 };
constexpr int kForkChunk = 256, kChunkEach = kForkChunk / 32;
__host__ __device__ constexpr int fork_chunks(int max_pages) {
  return max_pages > 0 ? (max_pages + kForkChunk - 1) / kForkChunk : 1;
}

template <int kPhase>
__global__ void __launch_bounds__(kPlanThreads, 1) fork_kernel(const ForkArgs a) {
  extern __shared__ int taken[];  // [B]: rows that take row r
  const PoolState& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = fork_chunks(s.max_pages);
  const long long items = (long long)s.B * chunks;
  const long long step = (long long)gridDim.x * kPlanWarps, first = (long long)blockIdx.x * kPlanWarps + warp;
  auto parent_of = [&](int b) {
    const int p = __ldg(a.parents + b);
    if (p < s.B) return p < 0 ? -1 : p;
    report(s);
    return b;
  };
  auto length = [&](int b) {  // before the fork
    const int L = s.lens[b];
    if (length_ok(s, L)) return L;
    report(s);
    return 0;
  };
  if constexpr (kPhase & kGather) {
    grid_dependents_launch();
    for (int b = threadIdx.x; b < s.B; b += kPlanThreads) taken[b] = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < s.B; b += kPlanThreads) {
      const int p = parent_of(b);
      if (p >= 0) atomicAdd(&taken[p], 1);
    }
    __syncthreads();
    for (long long item = first; item < items; item += step) {
      const int b = (int)(item / chunks), i0 = (int)(item - (long long)b * chunks) * kForkChunk + lane;
      const int c = taken[b], p = parent_of(b);
      const int L = length(b), n = c != 1 ? pages_of(s, L) : 0;
      const int32_t* row = s.table + (size_t)b * s.max_pages;
      int page[kChunkEach];
#pragma unroll
      for (int j = 0; j < kChunkEach; ++j) page[j] = i0 + 32 * j < n ? row[i0 + 32 * j] : -1;
#pragma unroll
      for (int j = 0; j < kChunkEach; ++j) add_refs(s, page[j], c - 1);
      if (p == b) continue;
      const int new_length = p < 0 ? 0 : length(p), m = pages_of(s, new_length);
      const int32_t* from = s.table + (size_t)(p < 0 ? 0 : p) * s.max_pages;
      int32_t* to = a.rows + (size_t)b * s.max_pages;
#pragma unroll
      for (int j = 0; j < kChunkEach; ++j) page[j] = i0 + 32 * j < m ? from[i0 + 32 * j] : -1;
#pragma unroll
      for (int j = 0; j < kChunkEach; ++j) {
        if (page[j] >= s.num_pages) report(s);
        if (i0 + 32 * j < m) to[i0 + 32 * j] = page[j];
      }
      if (i0 == 0) {
        a.old_lens[b] = L;
        a.new_lens[b] = new_length;
      }
    }
  }
  if constexpr (kPhase == kBoth) cluster_sync();
  if constexpr (kPhase == kScatter) grid_dependency_wait();
  if constexpr (kPhase & kScatter) {
    for (long long item = first; item < items; item += step) {
      const int b = (int)(item / chunks), i0 = (int)(item - (long long)b * chunks) * kForkChunk + lane;
      if (parent_of(b) == b) continue;
      const int L = __ldcg(a.new_lens + b), n = pages_of(s, L), old = pages_of(s, __ldcg(a.old_lens + b));
      int32_t* row = s.table + (size_t)b * s.max_pages;
      const int32_t* from = a.rows + (size_t)b * s.max_pages;
      int page[kChunkEach];
#pragma unroll
      for (int j = 0; j < kChunkEach; ++j) page[j] = i0 + 32 * j < n ? __ldcg(from + i0 + 32 * j) : -1;
#pragma unroll
      for (int j = 0; j < kChunkEach; ++j)
        if (i0 + 32 * j < (n > old ? n : old)) row[i0 + 32 * j] = page[j];
      if (i0 == 0) s.lens[b] = L;
    }
  }
}

// ---------------------------------------------------------------- resize
// Lengths of row b before and after; a bad length leaves the row as it is, no row at all has none.
struct RowLens {
  int L = 0, N = 0;
  bool ok = true;
  __device__ __forceinline__ RowLens(const ResizeArgs& a, int b, int end) {
    if (b >= end) return;
    L = a.s.lens[b];
    N = __ldg(a.new_lens + b);
    ok = length_ok(a.s, L) && length_ok(a.s, N);
    if (!ok) {
      if (!length_ok(a.s, L)) L = 0;
      N = L;
    }
  }
};

// Calls f(b, i, page) for the table entries that the warp's rows give back (lane l has row b0 + l):
// those behind a row's new length (empty ones too), and with a window those wholly below it, from
// the window's edge down to the next entry that holds no page. The warp takes its rows one by one;
// `subs` warps share the long way of a row.
constexpr int kWalk = 4;      // words of a row in flight
constexpr int kFewPages = 4;  // pages of a row that its lane sees to alone
template <class F>
__device__ __forceinline__ void released(const ResizeArgs& a, int b0, const RowLens& r, int lane, int sub, int subs,
                                         F f) {
  const PoolState& s = a.s;
  const int n0 = pages_of(s, r.N), n1 = pages_of(s, r.L);
  int top = -1;  // the last entry wholly below the lowest position that stays visible
  if (a.window > 0 && sub == 0) {
    const int low = imin(r.L, r.N) - a.window + 1;
    if (low > 0) top = page_index(s, low) - 1;
    if (top >= 0 && s.table[(size_t)(b0 + lane) * s.max_pages + top] < 0) top = -1;  // the usual case
  }
  const bool few = n1 - n0 <= kFewPages;  // by the row's own lane
  if (few && sub == 0)
    for (int i = n0; i < n1; ++i) f(b0 + lane, i, s.table[(size_t)(b0 + lane) * s.max_pages + i]);
#pragma unroll 1
  for (uint32_t todo = __ballot_sync(0xffffffffu, !few || top >= 0); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1, b = b0 + who;
    const int32_t* row = s.table + (size_t)b * s.max_pages;
    const int end = __shfl_sync(0xffffffffu, few ? n0 : n1, who);
#pragma unroll 4
    for (int i = __shfl_sync(0xffffffffu, n0, who) + lane + 32 * sub; i < end; i += 32 * subs) f(b, i, row[i]);
    bool more = true;
#pragma unroll 1
    for (int t = __shfl_sync(0xffffffffu, top, who) - lane; more; t -= 32 * kWalk) {
      int page[kWalk];
#pragma unroll
      for (int j = 0; j < kWalk; ++j) page[j] = t - 32 * j >= 0 ? row[t - 32 * j] : -1;
#pragma unroll
      for (int j = 0; j < kWalk; ++j) {
        const uint32_t holes = __ballot_sync(0xffffffffu, page[j] < 0);
        if (more && lane < (holes ? __ffs(holes) - 1 : 32)) f(b, t - 32 * j, page[j]);
        more = more && !holes;
      }
    }
  }
}

// Calls f(first page, mask of the free ones among 32 pages from there) for [lo, hi), kMasks words of
// counts in flight; f says whether to go on.
constexpr int kMasks = 8;
template <class F>
__device__ __forceinline__ void free_masks(const int32_t* refs, int lo, int hi, int lane, F f) {
#pragma unroll 1
  for (int p = lo; p < hi; p += 32 * kMasks) {
    uint32_t is_free = 0;
#pragma unroll
    for (int j = 0; j < kMasks; ++j) {
      const int at = p + 32 * j + lane;
      if (at < hi && __ldcg(refs + at) == 0) is_free |= 1u << j;
    }
#pragma unroll 1
    for (int j = 0; j < kMasks && p + 32 * j < hi; ++j)
      if (!f(p + 32 * j, __ballot_sync(0xffffffffu, is_free >> j & 1))) return;
  }
}

constexpr int kNoMove = -1, kFreshPage = -2;

__global__ void __launch_bounds__(kPlanThreads, 1) resize_kernel(const ResizeArgs a) {
  __shared__ unsigned long long scan[kPlanWarps];
  __shared__ Totals needs, move_counts, frees;
  __shared__ int warp_free[kPlanWarps];
  const PoolState& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_rank(), ctas = cluster_size();
  auto sync = [&] {
    if (ctas == 1) __syncthreads();
    else cluster_sync();
  };
  const Share rows(s.B, cta, ctas), mine(s.num_pages, cta * kPlanWarps + warp, ctas * kPlanWarps);
  // rows of a warp at a time, or warps of a row: long rows are spread over the warps
  const int n_rows = rows.hi - rows.lo;
  const int each = imax(1, imin(32, (n_rows + kPlanWarps - 1) / kPlanWarps));
  const int subs = imax(1, kPlanWarps / imax(1, n_rows)), sub = warp % subs;
  const int row0 = rows.lo + warp / subs * each, row_step = kPlanWarps / subs * each;
  grid_dependents_launch();

  // 1. what rows give back leaves the counts; the partial pages that rows will write into
  for (int b0 = row0; b0 < rows.hi; b0 += row_step) {
    const int b = b0 + lane, end = imin(b0 + each, rows.hi);
    const RowLens r(a, b, end);
    if (!r.ok) report(s);
    int page = kNoMove;
    if (sub == 0 && r.N > r.L && r.L % s.page_size != 0) {
      page = s.table[(size_t)b * s.max_pages + page_index(s, r.L)];
      if (page < 0 || page >= s.num_pages) {  // its tokens are nowhere: a new page, no copy
        report(s);
        page = kFreshPage;
      } else {
        a.writers[page] = 0;
        a.lowest[page] = s.B;
      }
    }
    if (sub == 0 && b < end) a.write_page[b] = page;
    released(a, b0, r, lane, sub, subs, [&](int, int, int page) { add_refs(s, page, -1); });
  }
  sync();

  // 2. the rows that write into a page that others hold too; the free pages
  for (int b = rows.lo + (int)threadIdx.x; b < rows.hi; b += kPlanThreads) {
    const int page = a.write_page[b];
    if (page >= 0 && __ldcg(s.refs + page) > 1) {
      atomicAdd(a.writers + page, 1);
      atomicMin(a.lowest + page, b);
    }
  }
  int n_free = 0;
  free_masks(s.refs, mine.lo, mine.hi, lane, [&](int, uint32_t m) {
    n_free += __popc(m);
    return true;
  });
  if (lane == 0) warp_free[warp] = n_free;
  sync();

  // 3. pages that each row needs. Of the g rows that write into a page with r holders all
  // take a copy if others hold it (r > g), else all but the lowest.
  unsigned long long need = 0, moves = 0;
  for (int b0 = rows.lo; b0 < rows.hi; b0 += kPlanThreads) {
    const int b = b0 + (int)threadIdx.x;
    unsigned long long n = 0, m = 0;
    int page = kNoMove;
    if (b < rows.hi) {
      const RowLens r(a, b, rows.hi);
      const int grown = pages_of(s, r.N) - pages_of(s, r.L);
      page = a.write_page[b];
      if (page >= 0) {
        const int holders = __ldcg(s.refs + page);
        if (holders > 1) m = holders > __ldcg(a.writers + page) || __ldcg(a.lowest + page) != b;
      }
      n = (unsigned long long)(grown > 0 ? grown : 0) + (page == kFreshPage) + m;
    }
    unsigned long long all;
    const unsigned long long at = block_scan(n | m << 48, scan, all), low = (1ull << 48) - 1;
    if (b < rows.hi) {
      a.row_rank[b] = (int)imin64((long long)(need + (at & low)), 0x7fffffff);
      a.row_move[b] = m ? (int)(moves + (at >> 48)) : page == kFreshPage ? kFreshPage : kNoMove;
    }
    need += all & low;
    moves += all >> 48;
  }
  if (warp == 0) {
    int f = warp_free[lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
    needs.publish(need, lane);
    move_counts.publish(moves, lane);
    frees.publish((unsigned long long)f, lane);
  }
  sync();

  // 4. all or nothing
  const unsigned long long need_all = needs.sum(), free_all = frees.sum();
  const bool lacking = need_all > free_all;
  if (cta == 0 && threadIdx.x == 0) {
    *a.missing = lacking ? (int)imin64((long long)(need_all - free_all), 0x7fffffff) : 0;
    *a.moves.count = lacking ? 0 : (int)move_counts.sum();
  }
  if (lacking) {
    for (int b0 = row0; b0 < rows.hi; b0 += row_step)
      released(a, b0, RowLens(a, b0 + lane, imin(b0 + each, rows.hi)), lane, sub, subs,
               [&](int, int, int page) { add_refs(s, page, 1); });
    return;
  }
  if (need_all > 0) {  // the lowest free pages, in order
    const int need_n = (int)need_all;
    int rank = (int)frees.before(cta);
    for (int w = 0; w < warp; ++w) rank += warp_free[w];
    if (rank < need_n)
      free_masks(s.refs, mine.lo, mine.hi, lane, [&](int p, uint32_t m) {
        const int at = rank + __popc(m & ((1u << lane) - 1));
        if ((m >> lane & 1) && at < need_n) {
          a.free_list[at] = p + lane;
          s.refs[p + lane] = 1;
        }
        rank += __popc(m);
        return rank < need_n;
      });
    sync();
  }

  // 5. the rows
  const int need0 = (int)needs.before(cta), move0 = (int)move_counts.before(cta);
  for (int b0 = row0; b0 < rows.hi; b0 += row_step) {
    const int b = b0 + lane;
    const RowLens r(a, b, imin(b0 + each, rows.hi));
    released(a, b0, r, lane, sub, subs, [&](int row, int i, int) { s.table[(size_t)row * s.max_pages + i] = -1; });
    int rank = 0, n0 = 0, n1 = 0;
    if (r.N > r.L) {
      const int move = a.row_move[b], fresh = move != kNoMove;
      rank = need0 + a.row_rank[b];
      int32_t* row = s.table + (size_t)b * s.max_pages;
      if (fresh && sub == 0) {
        const int page = __ldcg(a.free_list + rank);
        row[page_index(s, r.L)] = page;
        if (move >= 0) {
          const int from = a.write_page[b];
          atomicAdd(s.refs + from, -1);
          a.moves.src[move0 + move] = from;
          a.moves.dst[move0 + move] = page;
          a.moves.tokens[move0 + move] = r.L % s.page_size;
        }
      }
      rank += fresh;
      n0 = pages_of(s, r.L);
      n1 = pages_of(s, r.N);
      if (n1 - n0 <= kFewPages) {  // a decode step
        for (int i = n0; i < n1; ++i) row[i] = __ldcg(a.free_list + rank + (i - n0));
        n1 = n0;
      }
    }
#pragma unroll 1
    for (uint32_t todo = __ballot_sync(0xffffffffu, n1 > n0); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1, first = __shfl_sync(0xffffffffu, n0, who);
      const int count = __shfl_sync(0xffffffffu, n1, who) - first;
      const int32_t* pages = a.free_list + __shfl_sync(0xffffffffu, rank, who);
      int32_t* row = s.table + (size_t)(b0 + who) * s.max_pages + first;
#pragma unroll 4
      for (int i = lane + 32 * sub; i < count; i += 32 * subs) row[i] = __ldcg(pages + i);
    }
    if (subs == 1 && r.N != r.L) s.lens[b] = r.N;
  }
  if (subs == 1) return;
  __syncthreads();  // the row's other warps have read its length
  for (int b = rows.lo + (int)threadIdx.x; b < rows.hi; b += kPlanThreads) {
    const RowLens r(a, b, rows.hi);
    if (r.N != r.L) s.lens[b] = r.N;
  }
}

// ---------------------------------------------------------------- compact
// With U used pages, the k-th highest used page from U on moves to the k-th lowest free page
// below U: as many of the one kind as of the other.
__global__ void __launch_bounds__(kPlanThreads, 1) compact_kernel(const CompactArgs a) {
  __shared__ Totals used, holes;
  __shared__ int warp_used[kPlanWarps], warp_holes[kPlanWarps];
  const PoolState& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_rank(), ctas = cluster_size();
  grid_dependents_launch();
  cluster_started_arrive();
  const Share mine(s.num_pages, cta * kPlanWarps + warp, ctas * kPlanWarps);
  auto publish = [&](Totals& t, int* per_warp, int n) {
    if (lane == 0) per_warp[warp] = n;
    __syncthreads();
    if (warp == 0) {
      int f = per_warp[lane];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
      t.publish((unsigned long long)f, lane);
    }
    cluster_sync();
  };
  int n = 0;
  free_masks(s.refs, mine.lo, mine.hi, lane, [&](int p, uint32_t free) {
    const int in = imax(0, imin(32, mine.hi - p));
    n += in - __popc(free);
    return true;
  });
  cluster_started_wait();
  publish(used, warp_used, n);
  const int U = (int)used.sum();
  int rank = (int)used.before(cta), n_holes = 0;  // used pages before p
  for (int w = 0; w < warp; ++w) rank += warp_used[w];
  free_masks(s.refs, mine.lo, mine.hi, lane, [&](int p0, uint32_t free) {
    const int in = imax(0, imin(32, mine.hi - p0)), p = p0 + lane;
    const bool inside = lane < in, is_used = inside && !(free >> lane & 1);
    const int u = rank + lane - __popc(free & ((1u << lane) - 1));
    const bool hole = inside && !is_used && p < U;
    if (is_used && p >= U) a.moves.src[U - 1 - u] = p;
    else if (inside) a.page_map[p] = is_used ? p : -1;
    if (hole) a.moves.dst[p - u] = p;
    n_holes += __popc(__ballot_sync(0xffffffffu, hole));
    rank += in - __popc(free);
    return true;
  });
  publish(holes, warp_holes, n_holes);
  const int M = (int)holes.sum();
  if (cta == 0 && threadIdx.x == 0) {
    *a.used = U;
    *a.moves.count = M;
  }
  for (int k = cta * kPlanThreads + threadIdx.x; k < M; k += ctas * kPlanThreads) {
    const int src = __ldcg(a.moves.src + k), dst = __ldcg(a.moves.dst + k);
    a.page_map[src] = dst;
    s.refs[dst] = s.refs[src];
    s.refs[src] = 0;
  }
}

// A cluster's four barriers cost a resize 1-2 us, its CTAs speed up what rows have to give back and
// to take: 64 rows of a decode step over 8900 pages 9.8 us in one CTA, 10.9 in three or four; 160
// rows that end, start and go on over 18000 pages 13.3 in eight, 16.7 in two; over 99500 pages with
// a window 17.8 in sixteen, 25 in eight. A compaction has fewer barriers and more to do per page
// (8900 pages 11.8 us in eight CTAs, 13.4 in two).
constexpr int kResizeOne = 12288, kResizeEach = 4096;
constexpr int kCompactOne = 2048, kCompactEach = 2048;
constexpr int kForkOne = 16384, kForkEach = 16384;  // table entries

// `state`: two words of the launch site's kernel for large_clusters.
template <class Args>
cudaError_t launch_plan(void (*kernel)(const Args), const Args& a, int ctas, size_t smem, cudaStream_t st,
                        std::atomic<uint64_t>* state) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (ctas > kPortableCtas && !large_clusters((const void*)kernel, cfg, state[0], state[1])) {
    cfg.gridDim = dim3(kPortableCtas);
    attr[0].val.clusterDim.x = kPortableCtas;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_fork(const ForkArgs& a, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> done[3], large[2];
  const long long items = (long long)a.s.B * fork_chunks(a.s.max_pages);
  const size_t smem = (size_t)a.s.B * 4;
  cudaError_t e;
  if (items <= 4 * kPortableCtas * kPlanWarps) {
    if ((e = allow_smem((const void*)fork_kernel<kBoth>, kForkMaxRows * 4, done[0])) != cudaSuccess) return e;
    return launch_plan(fork_kernel<kBoth>, a, plan_ctas(items * kForkChunk, kForkOne, kForkEach), smem, st, large);
  }
  if ((e = allow_smem((const void*)fork_kernel<kGather>, kForkMaxRows * 4, done[1])) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(num_sms > 0 ? num_sms : 1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  if ((e = cudaLaunchKernelEx(&cfg, fork_kernel<kGather>, a)) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fork_kernel<kScatter>, a);
}

cudaError_t launch_resize(const ResizeArgs& a, const PageCopy& c, int num_sms, cudaStream_t st) {
  const long long work = imin64(0x7fffffff, (long long)a.s.num_pages + 16LL * a.s.B);
  static std::atomic<uint64_t> large[2];
  const cudaError_t e = launch_plan(resize_kernel, a, plan_ctas(work, kResizeOne, kResizeEach), 0, st, large);
  return e == cudaSuccess ? launch_page_copy(c, num_sms, st) : e;
}

cudaError_t launch_compact(const CompactArgs& a, const PageCopy& c, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> large[2];
  const cudaError_t e = launch_plan(compact_kernel, a, plan_ctas(a.s.num_pages, kCompactOne, kCompactEach), 0, st, large);
  return e == cudaSuccess ? launch_compact_copy(c, a, num_sms, st) : e;
}

}  // namespace attn
