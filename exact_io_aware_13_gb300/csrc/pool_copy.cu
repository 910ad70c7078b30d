// Copies of cache pages: the partial pages that a resize copies before they are written and the
// pages that a compaction moves (listed by the plan kernels of pool.cu), and pages copied between
// pools. A whole page is one run of Hkv * page_size rows per tensor, the first tokens of a page
// one run per kv head.
//
// Bound by HBM: every byte is read once and written once. Bulk copies carry a run in pieces of 8
// KB through shared memory, each warp with a ring of its own, so that 96 KB of loads and as much of
// stores per SM are in flight from one small CTA, which starts fast when there is nothing to copy.
// Measured: 1823 pages of 256 KB in 154 us (6.2 TB/s of reads and writes), half of 8660 such pages
// moved to the front in 169 us (6.3 TB/s); 16-byte loads of 256 threads took 40 us more there.
// Pieces of small pages, one per lane: 97656 pages of 2 KB per tensor in 155 us, 179 by the ring.
#include "paged.cuh"
#include "pool.cuh"

namespace attn {
namespace {

constexpr int kCopyWarps = 4;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kPiece = 8192;             // bytes
constexpr int kStages = 6, kInFlight = 3;  // pieces of a warp's ring, and loads ahead of the stores
constexpr int kCopySmem = kCopyWarps * kStages * kPiece;

constexpr int kSmallBelow = 4096;        // runs of fewer bytes: a piece per lane
constexpr int kSmallPiece = 768;
constexpr int kSmallSmem = kCopyWarps * 64 * kSmallPiece;

// kListed, kCompact: the moves of a plan kernel (a compaction rewrites the table too). kShort,
// kOwned: a caller's list, of up to kShortList entries or with its owners found before.
enum CopyMode { kListed, kCompact, kShort, kOwned };
constexpr int kShortList = 32;

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {  // at most N groups still read shared memory
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Table entries of the rows after a compaction.
__device__ void rewrite_table(const CompactArgs& c) {
  const PoolState& s = c.s;
  const int lane = threadIdx.x & 31;
  const int U = __ldcg(c.used);
  const int warps = gridDim.x * kCopyWarps;
  for (int b = blockIdx.x * kCopyWarps + (threadIdx.x >> 5); b < s.B; b += warps) {
    const int L = __ldg(s.lens + b);
    if (!length_ok(s, L)) {
      atomicOr(s.status, DEV_BAD_INPUT);
      continue;
    }
    int32_t* row = s.table + (size_t)b * s.max_pages;
#pragma unroll 4
    for (int i = lane, n = pages_of(s, L); i < n; i += 32) {
      const int page = row[i];
      if (page < U) continue;  // not moved, or no page
      const int to = page < s.num_pages ? __ldcg(c.page_map + page) : -1;
      if (to < 0) atomicOr(s.status, DEV_BAD_INPUT);
      else row[i] = to;
    }
  }
}

// An entry of a caller's list that names two pages.
__device__ __forceinline__ bool is_entry(const CopyList& l, int src, int dst) {
  return src >= 0 && dst >= 0 && src < l.num_pages_from && dst < l.num_pages_to;
}

// Whether a source page can be another entry's destination, and so has an owner (one pool may be
// described with two sizes).
__device__ __forceinline__ bool may_be_written(const CopyList& l, int src) {
  return l.same_pool && src < l.num_pages_to;
}

// The first entry with each destination. kInit: one CTA puts the owners that it meets back first
// (195 entries: 5.9 us with the copy, against 10.1 behind a memset of all owners, which many entries
// over all SMs take).
template <bool kInit>
__global__ void __launch_bounds__(1024) copy_owner_kernel(const CopyList l) {
  grid_dependents_launch();
  const int first = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  if constexpr (kInit) {
    for (int i = first; i < l.n; i += step) {
      const int src = __ldg(l.src + i), dst = __ldg(l.dst + i);
      if (!is_entry(l, src, dst)) continue;
      l.owner[dst] = 0x7fffffff;
      if (may_be_written(l, src)) l.owner[src] = 0x7fffffff;
    }
    __syncthreads();
  }
  for (int i = first; i < l.n; i += step) {
    const int src = __ldg(l.src + i), dst = __ldg(l.dst + i);
    if (is_entry(l, src, dst)) atomicMin(l.owner + dst, i);
    else if (src >= l.num_pages_from || dst >= l.num_pages_to) atomicOr(l.status, DEV_BAD_INPUT);
  }
}
constexpr int kOneCtaList = 1024;

// The entries of a short list that are copied, one per lane.
__device__ __forceinline__ void check_list(const CopyList& p, int* src, int* dst) {
  const int i = threadIdx.x;
  if (i < 32) {
    const int from = i < p.n ? __ldg(p.src + i) : -1, to = i < p.n ? __ldg(p.dst + i) : -1;
    const bool outside = from >= p.num_pages_from || to >= p.num_pages_to;
    bool ok = is_entry(p, from, to);
    const bool entry = ok;
    const uint32_t same = __match_any_sync(0xffffffffu, entry ? to : -1 - i);
    ok = ok && (same & ((1u << i) - 1)) == 0;
    if (p.same_pool)
      for (int j = 0; j < p.n; ++j) {
        const int other = __shfl_sync(0xffffffffu, entry ? to : -1, j);
        ok = ok && (j == i || from == to || other != from);
      }
    if ((entry && !ok) || outside) atomicOr(p.status, DEV_BAD_INPUT);
    src[i] = ok && !(p.same_pool && from == to) ? from : -1;
    dst[i] = to;
  }
  __syncthreads();
}

// A list of moves cut into pieces of kBytes: which bytes piece u copies.
struct Piece {
  const uint8_t* from;
  uint8_t* to;
  int n;  // bytes, a multiple of 2, 0: nothing; both addresses 16-byte aligned
};
template <int kBytes, CopyMode kMode>
struct Pieces {
  const PageCopy& c;
  const CopyList& given;
  const int *src, *dst;
  int bytes_kv;  // of a token and head
  int per_run, per_move;
  long long count, page_rows;
  __device__ __forceinline__ Pieces(const PageCopy& c_, const CopyList& given_, const int* src_, const int* dst_,
                                    int moves)
      : c(c_), given(given_), src(src_), dst(dst_), bytes_kv(c_.e4m3 ? c_.d : 2 * c_.d), per_run(2 * c_.kv_pieces + c_.exp_pieces),
        per_move(c_.runs * per_run), count((long long)moves * per_move),
        page_rows((long long)c_.Hkv * c_.page_size) {}
  __device__ __forceinline__ Piece get(long long u) const {
    Piece x{nullptr, nullptr, 0};
    if (u >= count) return x;
    int move, rest;
    if (u < 0x7fffffff) {
      move = (int)((unsigned)u / (unsigned)per_move);
      rest = (int)u - move * per_move;
    } else {
      move = (int)(u / per_move);
      rest = (int)(u - (long long)move * per_move);
    }
    const int s = kMode == kShort ? src[move] : __ldcg(src + move), d = kMode == kShort ? dst[move] : __ldcg(dst + move);
    if (s < 0) return x;
    if constexpr (kMode == kOwned) {
      if (!is_entry(given, s, d)) return x;
      const bool itself = given.same_pool && s == d;
      if (__ldcg(given.owner + d) != move || (may_be_written(given, s) && !itself && __ldcg(given.owner + s) < given.n)) {
        atomicOr(given.status, DEV_BAD_INPUT);
        return x;
      }
      if (itself) return x;
    }
    const int run = c.runs > 1 ? rest / per_run : 0, part = rest - run * per_run;
    const int which = part < c.kv_pieces ? 0 : part < 2 * c.kv_pieces ? 1 : 2;
    const int bytes = which == 2 ? 2 : bytes_kv;
    const long long tokens = c.moves.tokens ? (long long)__ldcg(c.moves.tokens + move) : page_rows;
    const long long at = (long long)(part - which * c.kv_pieces) * kBytes;
    const long long off = (long long)run * c.page_size * bytes + at, page = page_rows * bytes;
    const long long left = tokens * bytes - at;
    if (left <= 0) return x;
    x.n = (int)imin64(left, kBytes);
    const void* from = which == 0 ? c.from[0] : which == 1 ? c.from[1] : c.from[2];
    void* to = which == 0 ? c.to[0] : which == 1 ? c.to[1] : c.to[2];
    x.from = static_cast<const uint8_t*>(from) + s * page + off;
    x.to = static_cast<uint8_t*>(to) + d * page + off;
    return x;
  }
};

// The tail of a piece behind its whole 16-byte words (partial pages' scales).
__device__ __forceinline__ void copy_tail(const Piece& x, int i) {
  const int whole = x.n & ~15;
  if (i < (x.n - whole) / 2)
    reinterpret_cast<uint16_t*>(x.to + whole)[i] = reinterpret_cast<const uint16_t*>(x.from + whole)[i];
}

// The moves to copy, once they are known: their number, and where their pages stand.
template <CopyMode kMode>
__device__ __forceinline__ int moves_of(const PageCopy& c, const CompactArgs& compact, const CopyList& given,
                                        int* list, const int*& src, const int*& dst) {
  if constexpr (kMode == kShort) {
    check_list(given, list, list + kShortList);
    src = list;
    dst = list + kShortList;
    return given.n;
  } else if constexpr (kMode == kOwned) {
    grid_dependency_wait();
    src = given.src;
    dst = given.dst;
    return given.n;
  } else {
    grid_dependency_wait();
    if constexpr (kMode == kCompact) rewrite_table(compact);
    src = c.moves.src;
    dst = c.moves.dst;
    return __ldcg(c.moves.count);
  }
}

// Small pages: a piece per lane. The 32 loads of a batch complete on one barrier; the next batch is
// on its way while a batch is stored. (Not for short lists, which have few pieces.)
template <CopyMode kMode>
__global__ void __launch_bounds__(kCopyThreads) small_copy_kernel(const PageCopy c, const CompactArgs compact,
                                                                 const CopyList given) {
  static_assert(kMode != kShort, "");
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ __align__(8) uint64_t full[kCopyWarps * 2];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(full + warp * 2);
  const uint32_t slot = smem_u32(ring_smem) + (warp * 64 + lane) * kSmallPiece;  // + 32 * kSmallPiece: odd batches
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane < 2) mbar_init(bar + lane * 8, 1);
  fence_barrier_init();
  __syncthreads();
  const int *src, *dst;
  const int moves = moves_of<kMode>(c, compact, given, nullptr, src, dst);
  if (moves == 0) return;
  const WaitCtx wait{&abort_flag, c.status};
  const Pieces<kSmallPiece, kMode> pieces(c, given, src, dst, moves);
  const long long units = pieces.count, stride = (long long)gridDim.x * kCopyThreads;
  auto load = [&](long long u, int k) {  // batch k
    const Piece x = pieces.get(u + lane);
    const int whole = x.n & ~15;
    int sum = whole;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const uint32_t b = bar + (k & 1) * 8;
    if (lane == 0) mbar_arrive_expect_tx(b, sum);
    __syncwarp();
    if (whole > 0) bulk_load(slot + (k & 1) * 32 * kSmallPiece, x.from, whole, b);
    for (int j = 0; 2 * j < x.n - whole; ++j) copy_tail(x, j);
    return x;
  };
  long long u = ((long long)blockIdx.x * kCopyWarps + warp) * 32;
  bool ok = u < units;
  Piece x{nullptr, nullptr, 0};
  if (ok) x = load(u, 0);
#pragma unroll 1
  for (int k = 0; ok; ++k) {
    u += stride;
    Piece next{nullptr, nullptr, 0};
    const bool more = u < units;
    if (more) {
      bulk_wait_read<0>();  // (the store of batch k - 1 has left the slot)
      next = load(u, k + 1);
    }
    const uint32_t b = bar + (k & 1) * 8;
    ok = __all_sync(0xffffffffu, mbar_wait(b, (k >> 1) & 1, wait));
    if (!ok) {
      drain_wait(b, (k >> 1) & 1);
      if (more) drain_wait(bar + ((k + 1) & 1) * 8, ((k + 1) >> 1) & 1);
      break;
    }
    if (x.n >= 16) bulk_store(x.to, slot + (k & 1) * 32 * kSmallPiece, x.n & ~15);
    bulk_commit();
    x = next;
    ok = more;
  }
  bulk_wait_all();
}

template <CopyMode kMode>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageCopy c, const CompactArgs compact,
                                                                const CopyList given) {
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ __align__(8) uint64_t full[kCopyWarps * kStages];
  __shared__ uint8_t* to_of[kCopyWarps][kStages];  // where a stage's piece goes
  __shared__ int n_of[kCopyWarps][kStages];
  __shared__ int abort_flag;
  __shared__ int list[kMode == kShort ? 2 * kShortList : 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(full + warp * kStages), ring = smem_u32(ring_smem) + warp * kStages * kPiece;
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane < kStages) mbar_init(bar + lane * 8, 1);
  fence_barrier_init();
  __syncthreads();
  const int *src, *dst;
  const int moves = moves_of<kMode>(c, compact, given, list, src, dst);
  if (moves == 0) return;
  const WaitCtx wait{&abort_flag, c.status};
  const Pieces<kPiece, kMode> pieces(c, given, src, dst, moves);
  const long long units = pieces.count, stride = (long long)gridDim.x * kCopyWarps;
  // Piece k of the warp goes through stage k % kStages; its store is issued kInFlight pieces after
  // its load. The lanes look 32 units up at a time; lane 0 issues, and it alone waits.
  int k = 0;
  bool ok = true;
  auto retire = [&](int j) {
    const int stage = j % kStages;
    const uint32_t b = bar + stage * 8, parity = (j / kStages) & 1;
    if (ok) ok = mbar_wait(b, parity, wait);
    if (ok) bulk_store(to_of[warp][stage], ring + stage * kPiece, n_of[warp][stage]);
    else drain_wait(b, parity);
    bulk_commit();
  };
#pragma unroll 1
  for (long long u = (long long)blockIdx.x * kCopyWarps + warp; u < units; u += 32 * stride) {
    const Piece mine = pieces.get(u + lane * stride);
#pragma unroll 1
    for (uint32_t todo = __ballot_sync(0xffffffffu, mine.n > 0); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1, n = __shfl_sync(0xffffffffu, mine.n, who), whole = n & ~15;
      const uint8_t* from = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.from), who));
      uint8_t* to = reinterpret_cast<uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.to), who));
      copy_tail(Piece{from, to, n}, lane);
      if (whole == 0) continue;
      if (lane == 0 && ok) {
        if (k >= kInFlight) retire(k - kInFlight);
        bulk_wait_read<kStages - kInFlight>();  // the store of piece k - kStages has left its stage
        const int stage = k % kStages;
        to_of[warp][stage] = to;
        n_of[warp][stage] = whole;
        mbar_arrive_expect_tx(bar + stage * 8, whole);
        bulk_load(ring + stage * kPiece, from, whole, bar + stage * 8);
        ++k;
      }
    }
  }
  if (lane == 0) {
    for (int j = k > kInFlight ? k - kInFlight : 0; j < k; ++j) retire(j);
    bulk_wait_all();
  }
}

template <CopyMode kMode>
cudaError_t launch(const PageCopy& copy, const CompactArgs& compact, const CopyList& given, long long most,
                   long long more_ctas, int num_sms, cudaStream_t st) {
  // Runs and pieces of a move: whole pages, or the first tokens of each head.
  PageCopy c = copy;
  c.runs = c.moves.tokens ? c.Hkv : 1;
  const long long tokens = c.moves.tokens ? c.page_size : (long long)c.Hkv * c.page_size;
  const long long kv = tokens * (c.e4m3 ? c.d : 2 * c.d);
  const long long exps = c.e4m3 ? tokens * 2 : 0, sms = num_sms > 0 ? num_sms : 1;
  auto pieces = [&](int piece) {
    // (the entries of pages without bytes are checked too, each by a piece of none)
    c.kv_pieces = kMode == kOwned && kv == 0 ? 1 : (int)((kv + piece - 1) / piece);
    c.exp_pieces = (int)((exps + piece - 1) / piece);
    return most * c.runs * (2 * c.kv_pieces + c.exp_pieces);
  };
  // Small pieces one per lane, unless there are few for a warp: then the ring's shorter way counts
  // (24 pages of 4 KB 3.3 us, a piece per lane 5.0).
  long long units = pieces(kPiece);
  bool small = false;
  auto kernel = page_copy_kernel<kMode>;
  if constexpr (kMode != kShort) {
    small = kv < kSmallBelow && units > 16 * kCopyWarps * sms;
    if (small) {
      units = pieces(kSmallPiece);
      kernel = small_copy_kernel<kMode>;
    }
  }
  const int smem = small ? kSmallSmem : kCopySmem;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem((const void*)kernel, smem, done[small]);
  if (e != cudaSuccess) return e;
  const int per_cta = small ? kCopyThreads : kCopyWarps;
  const long long ctas = (units + per_cta - 1) / per_cta + more_ctas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)imin64(ctas > 0 ? ctas : 1, sms));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kMode == kShort ? 0 : 1;  // the others follow the kernel that lists their moves
  return cudaLaunchKernelEx(&cfg, kernel, c, compact, given);
}

}  // namespace

cudaError_t launch_page_copy(const PageCopy& c, int num_sms, cudaStream_t st) {
  return launch<kListed>(c, CompactArgs{}, CopyList{}, c.moves.most, 0, num_sms, st);
}
cudaError_t launch_compact_copy(const PageCopy& c, const CompactArgs& compact, int num_sms, cudaStream_t st) {
  // (the CTAs rewrite the table's rows too)
  return launch<kCompact>(c, compact, CopyList{}, c.moves.most, imin64(compact.s.B / kCopyWarps, num_sms), num_sms, st);
}
cudaError_t launch_copy_pages(const CopyList& l, const PageCopy& c, int num_sms, cudaStream_t st) {
  if (l.n <= kShortList) return launch<kShort>(c, CompactArgs{}, l, l.n, 0, num_sms, st);
  cudaError_t e = cudaSuccess;
  if (l.n <= kOneCtaList) {
    copy_owner_kernel<true><<<1, 1024, 0, st>>>(l);
  } else {
    e = cudaMemsetAsync(l.owner, 0x7f, (size_t)l.num_pages_to * 4, st);  // (above every entry)
    if (e != cudaSuccess) return e;
    const long long ctas = imin64((l.n + 255) / 256, 4LL * (num_sms > 0 ? num_sms : 1));
    copy_owner_kernel<false><<<(unsigned)ctas, 256, 0, st>>>(l);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch<kOwned>(c, CompactArgs{}, l, l.n, 0, num_sms, st);
}

}  // namespace attn
