// Plans of the pool's operators: who holds which page after a fork, a resize or a compaction,
// and which pages have to be copied for it (pool_copy.cu copies them).
//
// Everything here is integer work with one answer: free pages are handed out in ascending
// order, rows take them in order, and counters are sums, so no order of atomics shows. Each
// plan reads the counts of all pages at most twice (4 bytes a page) and the table entries that
// change; it is bound by the latency of its few steps, not by bytes.
#include "paged.cuh"
#include "pool.cuh"

namespace attn {
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
// its pages. The new rows are gathered into the workspace before any row is overwritten.
__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const ForkArgs a) {
  extern __shared__ int taken[];  // [B]: rows that take row r
  const PoolState& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = cluster_size() * kPlanWarps, first = cluster_rank() * kPlanWarps + warp;
  for (int b = threadIdx.x; b < s.B; b += kPlanThreads) taken[b] = 0;
  __syncthreads();
  auto parent_of = [&](int b) {
    const int p = __ldg(a.parents + b);
    if (p < s.B) return p < 0 ? -1 : p;
    report(s);
    return b;
  };
  for (int b = threadIdx.x; b < s.B; b += kPlanThreads) {
    const int p = parent_of(b);
    if (p >= 0) atomicAdd(&taken[p], 1);
  }
  __syncthreads();
  auto held = [&](int b) {  // pages of row b before the fork
    const int L = s.lens[b];
    if (length_ok(s, L)) return pages_of(s, L);
    report(s);
    return 0;
  };
  for (int b = first; b < s.B; b += step) {
    const int32_t* row = s.table + (size_t)b * s.max_pages;
    const int c = taken[b];
    if (c != 1)
      for (int i = lane, n = held(b); i < n; i += 32) add_refs(s, row[i], c - 1);
    const int p = parent_of(b);
    if (p == b) continue;
    const int n = p < 0 ? 0 : held(p);
    const int32_t* from = s.table + (size_t)(p < 0 ? 0 : p) * s.max_pages;
    int32_t* to = a.rows + (size_t)b * s.max_pages;
    for (int i = lane; i < n; i += 32) {
      const int page = from[i];
      if (page >= s.num_pages) report(s);
      to[i] = page;
    }
    if (lane == 0) a.lens[b] = n > 0 ? s.lens[p] : 0;
  }
  cluster_sync();
  for (int b = first; b < s.B; b += step) {
    if (parent_of(b) == b) continue;
    const int old = held(b), L = __ldcg(a.lens + b), n = pages_of(s, L);
    __syncwarp();
    int32_t* row = s.table + (size_t)b * s.max_pages;
    const int32_t* from = a.rows + (size_t)b * s.max_pages;
    for (int i = lane; i < n; i += 32) row[i] = __ldcg(from + i);
    for (int i = n + lane; i < old; i += 32) row[i] = -1;
    if (lane == 0) s.lens[b] = L;
  }
}

// ---------------------------------------------------------------- resize
// Lengths of row b before and after; a bad length leaves the row as it is.
struct RowLens {
  int L, N;
  __device__ __forceinline__ RowLens(const ResizeArgs& a, int b) {
    L = a.s.lens[b];
    N = __ldg(a.new_lens + b);
    if (!length_ok(a.s, L)) L = N = 0;
    if (!length_ok(a.s, N)) N = L;
  }
};

// Calls f(i, page) for the table entries that row b gives back, all lanes of a warp together:
// those behind its new length (empty ones too), and with a window those wholly below it, from
// the window's edge down to the next entry that holds no page.
template <class F>
__device__ __forceinline__ void released(const ResizeArgs& a, int b, const RowLens& r, int lane, F f) {
  const PoolState& s = a.s;
  const int32_t* row = s.table + (size_t)b * s.max_pages;
  for (int i = pages_of(s, r.N) + lane, n = pages_of(s, r.L); i < n; i += 32) f(i, row[i]);
  if (a.window <= 0) return;
  const int low = imin(r.L, r.N) - a.window + 1;  // the lowest position that stays visible
  for (int top = low > 0 ? page_index(s, low) - 1 : -1; top >= 0; top -= 32) {
    const int i = top - lane;
    const int page = i >= 0 ? row[i] : -1;
    const uint32_t holes = __ballot_sync(0xffffffffu, page < 0);
    if (lane < (holes ? __ffs(holes) - 1 : 32)) f(i, page);
    if (holes) break;
  }
}

constexpr int kNoMove = -1, kFreshPage = -2;

__global__ void __launch_bounds__(kPlanThreads) resize_kernel(const ResizeArgs a) {
  __shared__ unsigned long long scan[kPlanWarps];
  __shared__ Totals needs, move_counts, frees;
  __shared__ int warp_free[kPlanWarps];
  const PoolState& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_rank(), ctas = cluster_size();
  const Share rows(s.B, cta, ctas);
  grid_dependents_launch();

  // 1. what rows give back leaves the counts; the partial pages that rows will write into
  for (int b = rows.lo + warp; b < rows.hi; b += kPlanWarps)
    released(a, b, RowLens(a, b), lane, [&](int, int page) { add_refs(s, page, -1); });
  for (int b = rows.lo + (int)threadIdx.x; b < rows.hi; b += kPlanThreads) {
    const RowLens r(a, b);
    if (!length_ok(s, s.lens[b]) || !length_ok(s, __ldg(a.new_lens + b))) report(s);
    int page = kNoMove;
    if (r.N > r.L && r.L % s.page_size != 0) {
      page = s.table[(size_t)b * s.max_pages + page_index(s, r.L)];
      if (page < 0 || page >= s.num_pages) {  // its tokens are nowhere: a new page, no copy
        report(s);
        page = kFreshPage;
      }
    }
    a.write_page[b] = page;
  }
  cluster_sync();

  // 2. pages that each row needs. Of the g rows that write into a page with r holders all
  // take a copy if others hold it (r > g), else all but the lowest.
  unsigned long long need = 0, moves = 0;
  for (int b0 = rows.lo; b0 < rows.hi; b0 += kPlanThreads) {
    const int b = b0 + (int)threadIdx.x;
    unsigned long long n = 0, m = 0;
    if (b < rows.hi) {
      const RowLens r(a, b);
      const int page = __ldcg(a.write_page + b);
      const int grown = pages_of(s, r.N) - pages_of(s, r.L);
      n = (unsigned long long)(grown > 0 ? grown : 0);
      if (page == kFreshPage) {
        ++n;
      } else if (page >= 0) {
        const int holders = __ldcg(s.refs + page);
        if (holders > 1) {
          int g = 0, lowest = b;
          for (int x = 0; x < s.B; ++x)
            if (__ldcg(a.write_page + x) == page) {
              ++g;
              lowest = imin(lowest, x);
            }
          m = holders > g || lowest != b;
          n += m;
        }
      }
    }
    unsigned long long n_all, m_all;
    const unsigned long long n_at = block_scan(n, scan, n_all), m_at = block_scan(m, scan, m_all);
    if (b < rows.hi) {
      a.row_rank[b] = (int)imin64((long long)(need + n_at), 0x7fffffff);
      if (m) a.row_move[b] = (int)(moves + m_at);
      else a.row_move[b] = __ldcg(a.write_page + b) == kFreshPage ? kFreshPage : kNoMove;
    }
    need += n_all;
    moves += m_all;
  }
  // free pages of each warp's share of the pool
  const Share mine(s.num_pages, cta * kPlanWarps + warp, ctas * kPlanWarps);
  int n_free = 0;
  for (int p = mine.lo + lane; p - lane < mine.hi; p += 32)
    n_free += __popc(__ballot_sync(0xffffffffu, p < mine.hi && __ldcg(s.refs + p) == 0));
  if (lane == 0) warp_free[warp] = n_free;
  __syncthreads();
  if (warp == 0) {
    int f = warp_free[lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) f += __shfl_xor_sync(0xffffffffu, f, off);
    needs.publish(need, lane);
    move_counts.publish(moves, lane);
    frees.publish((unsigned long long)f, lane);
  }
  cluster_sync();

  // 3. all or nothing
  const unsigned long long need_all = needs.sum(), free_all = frees.sum();
  const bool lacking = need_all > free_all;
  if (cta == 0 && threadIdx.x == 0) {
    *a.missing = lacking ? (int)imin64((long long)(need_all - free_all), 0x7fffffff) : 0;
    *a.moves.count = lacking ? 0 : (int)move_counts.sum();
  }
  if (lacking) {
    for (int b = rows.lo + warp; b < rows.hi; b += kPlanWarps)
      released(a, b, RowLens(a, b), lane, [&](int, int page) { add_refs(s, page, 1); });
    return;
  }
  if (need_all > 0) {  // the lowest free pages, in order
    unsigned long long rank = frees.before(cta);
    for (int w = 0; w < warp; ++w) rank += warp_free[w];
    for (int p = mine.lo + lane; p - lane < mine.hi && rank < need_all; p += 32) {
      const bool is_free = p < mine.hi && __ldcg(s.refs + p) == 0;
      const uint32_t m = __ballot_sync(0xffffffffu, is_free);
      const unsigned long long at = rank + __popc(m & ((1u << lane) - 1));
      if (is_free && at < need_all) {
        a.free_list[at] = p;
        s.refs[p] = 1;
      }
      rank += __popc(m);
    }
    cluster_sync();
  }

  // 4. the rows
  const int need0 = (int)needs.before(cta), move0 = (int)move_counts.before(cta);
  for (int b = rows.lo + warp; b < rows.hi; b += kPlanWarps) {
    const RowLens r(a, b);
    int32_t* row = s.table + (size_t)b * s.max_pages;
    released(a, b, r, lane, [&](int i, int) { row[i] = -1; });
    const int move = a.row_move[b], fresh = move != kNoMove;
    const int32_t* pages = a.free_list + need0 + a.row_rank[b];
    for (int i = pages_of(s, r.L) + lane, j = fresh + lane, n = pages_of(s, r.N); i < n; i += 32, j += 32)
      row[i] = __ldcg(pages + j);
    if (lane == 0 && fresh) {
      const int page = __ldcg(pages);
      row[page_index(s, r.L)] = page;
      if (move >= 0) {
        const int from = a.write_page[b];
        atomicAdd(s.refs + from, -1);
        a.moves.src[move0 + move] = from;
        a.moves.dst[move0 + move] = page;
        a.moves.tokens[move0 + move] = r.L % s.page_size;
      }
    }
    __syncwarp();
    if (lane == 0 && r.N != r.L) s.lens[b] = r.N;
  }
}

// ---------------------------------------------------------------- compact
// With U used pages, the k-th highest used page from U on moves to the k-th lowest free page
// below U: as many of the one kind as of the other.
__global__ void __launch_bounds__(kPlanThreads) compact_kernel(const CompactArgs a) {
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
  for (int p = mine.lo + lane; p - lane < mine.hi; p += 32)
    n += __popc(__ballot_sync(0xffffffffu, p < mine.hi && s.refs[p] != 0));
  cluster_started_wait();
  publish(used, warp_used, n);
  const int U = (int)used.sum();
  int rank = (int)used.before(cta), n_holes = 0;  // used pages before p
  for (int w = 0; w < warp; ++w) rank += warp_used[w];
  for (int p = mine.lo + lane; p - lane < mine.hi; p += 32) {
    const bool in = p < mine.hi, is_used = in && s.refs[p] != 0;
    const uint32_t m = __ballot_sync(0xffffffffu, is_used);
    const int u = rank + __popc(m & ((1u << lane) - 1));
    const bool hole = in && !is_used && p < U;
    if (is_used && p >= U) a.moves.src[U - 1 - u] = p;
    else if (in) a.page_map[p] = is_used ? p : -1;
    if (hole) a.moves.dst[p - u] = p;
    n_holes += __popc(__ballot_sync(0xffffffffu, hole));
    rank += __popc(m);
  }
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

// ---------------------------------------------------------------- copy
// Of the entries with one destination the first is copied; within one pool an entry whose
// source is another's destination is not. The entries left out are reported.
__global__ void __launch_bounds__(kPlanThreads) copy_plan_kernel(const CopyPlanArgs a) {
  grid_dependents_launch();
  const int first = cluster_rank() * kPlanThreads + threadIdx.x, step = cluster_size() * kPlanThreads;
  auto entry = [&](int i, int& src, int& dst) {  // false: nothing to copy
    src = __ldg(a.src + i);
    dst = __ldg(a.dst + i);
    return src >= 0 && dst >= 0 && src < a.num_pages_from && dst < a.num_pages_to;
  };
  int src, dst;
  for (int i = first; i < a.n; i += step)
    if (entry(i, src, dst)) {
      a.owner[dst] = 0x7fffffff;
      if (a.same_pool) a.owner[src] = 0x7fffffff;
    } else if (src >= a.num_pages_from || dst >= a.num_pages_to) {
      atomicOr(a.status, DEV_BAD_INPUT);
    }
  cluster_sync();
  for (int i = first; i < a.n; i += step)
    if (entry(i, src, dst)) atomicMin(a.owner + dst, i);
  cluster_sync();
  for (int i = first; i < a.n; i += step) {
    bool copied = entry(i, src, dst);
    if (copied) {
      copied = __ldcg(a.owner + dst) == i;
      if (a.same_pool && src != dst && __ldcg(a.owner + src) != 0x7fffffff) copied = false;
      if (!copied) atomicOr(a.status, DEV_BAD_INPUT);
    }
    a.moves.src[i] = copied && !(a.same_pool && src == dst) ? src : -1;
    a.moves.dst[i] = dst;
  }
  if (first == 0) *a.moves.count = a.n;
}

// CTAs of a plan: one per 8192 units of work (pages or entries), as a power of two.
int plan_ctas(long long work) {
  int n = 1;
  while (n < kPlanMaxCtas && (long long)n * 8192 < work) n *= 2;
  return n;
}

template <class Args>
cudaError_t launch_plan(void (*kernel)(const Args), const Args& a, int ctas, size_t smem, cudaStream_t st) {
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
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem((const void*)fork_kernel, kForkMaxRows * 4, done);
  if (e != cudaSuccess) return e;
  return launch_plan(fork_kernel, a, plan_ctas((long long)a.s.B * a.s.max_pages), (size_t)a.s.B * 4, st);
}

cudaError_t launch_resize(const ResizeArgs& a, const PageCopy& c, int num_sms, cudaStream_t st) {
  const long long work = imin64(0x7fffffff, (long long)a.s.num_pages + 32LL * a.s.B);
  const cudaError_t e = launch_plan(resize_kernel, a, plan_ctas(work), 0, st);
  return e == cudaSuccess ? launch_page_copy(c, nullptr, num_sms, st) : e;
}

cudaError_t launch_compact(const CompactArgs& a, const PageCopy& c, int num_sms, cudaStream_t st) {
  const cudaError_t e = launch_plan(compact_kernel, a, plan_ctas(a.s.num_pages), 0, st);
  return e == cudaSuccess ? launch_page_copy(c, &a, num_sms, st) : e;
}

cudaError_t launch_copy_pages(const CopyPlanArgs& a, const PageCopy& c, int num_sms, cudaStream_t st) {
  const cudaError_t e = launch_plan(copy_plan_kernel, a, plan_ctas(a.n), 0, st);
  return e == cudaSuccess ? launch_page_copy(c, nullptr, num_sms, st) : e;
}

}  // namespace attn
