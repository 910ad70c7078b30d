// Copies of cache pages: the partial pages that a resize copies before they are written and the
// pages that a compaction moves (listed by the plan kernels of pool.cu), and pages copied between
// pools. A whole page is one run of Hkv * page_size rows per tensor, the first tokens of a page
// one run per kv head.
//
// Bound by HBM: every byte is read once and written once. Bulk copies carry a run in pieces of 8
// KB through shared memory, each warp with a ring of its own, so that 128 KB per SM are in flight
// from one small CTA, which starts fast when there is nothing to copy.
#include "paged.cuh"
#include "pool.cuh"

namespace attn {
namespace {

constexpr int kCopyWarps = 4;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kPiece = 8192;             // bytes
constexpr int kStages = 6, kInFlight = 3;  // pieces of a warp's ring, and loads ahead of the stores
constexpr int kCopySmem = kCopyWarps * kStages * kPiece;

enum CopyMode { kListed, kCompact, kDirect };

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

// The entries of a short list of the caller's that are copied (see copy_plan_kernel).
__device__ void check_list(const CopyPlanArgs& p, int* src, int* dst) {
  for (int i = threadIdx.x; i < p.n; i += kCopyThreads) {
    src[i] = __ldg(p.src + i);
    dst[i] = __ldg(p.dst + i);
  }
  __syncthreads();
  bool copied[(kCopyDirect + kCopyThreads - 1) / kCopyThreads];
#pragma unroll
  for (int k = 0; k < (kCopyDirect + kCopyThreads - 1) / kCopyThreads; ++k) {
    const int i = threadIdx.x + k * kCopyThreads;
    copied[k] = false;
    if (i >= p.n || src[i] < 0 || dst[i] < 0) {
      if (i < p.n && (src[i] >= p.num_pages_from || dst[i] >= p.num_pages_to)) atomicOr(p.status, DEV_BAD_INPUT);
      continue;
    }
    bool ok = src[i] < p.num_pages_from && dst[i] < p.num_pages_to;
    for (int j = 0; j < p.n && ok; ++j) {
      if (j == i || src[j] < 0 || dst[j] < 0 || src[j] >= p.num_pages_from || dst[j] >= p.num_pages_to) continue;
      ok = !(j < i && dst[j] == dst[i]) && !(p.same_pool && src[i] != dst[i] && dst[j] == src[i]);
    }
    if (!ok) atomicOr(p.status, DEV_BAD_INPUT);
    copied[k] = ok && !(p.same_pool && src[i] == dst[i]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < (kCopyDirect + kCopyThreads - 1) / kCopyThreads; ++k) {
    const int i = threadIdx.x + k * kCopyThreads;
    if (i < p.n && !copied[k]) src[i] = -1;
  }
  __syncthreads();
}

// What a unit of work copies; n = 0: nothing.
struct Unit {
  const uint8_t* from;
  uint8_t* to;
  int n;  // bytes, a multiple of 2; both addresses 16-byte aligned
};

template <CopyMode kMode>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageCopy c, const CompactArgs compact,
                                                                const CopyPlanArgs plan) {
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ __align__(8) uint64_t full[kCopyWarps * kStages];
  __shared__ uint8_t* to_of[kCopyWarps][kStages];  // where a stage's piece goes
  __shared__ int n_of[kCopyWarps][kStages];
  __shared__ int abort_flag;
  __shared__ int list[kMode == kDirect ? 2 * kCopyDirect : 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bar = smem_u32(full + warp * kStages), ring = smem_u32(ring_smem) + warp * kStages * kPiece;
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane < kStages) mbar_init(bar + lane * 8, 1);
  fence_barrier_init();
  __syncthreads();
  int count;
  if constexpr (kMode == kDirect) {
    count = plan.n;
    check_list(plan, list, list + kCopyDirect);
  } else {
    grid_dependency_wait();
    if constexpr (kMode == kCompact) rewrite_table(compact);
    count = __ldcg(c.moves.count);
  }
  if (count == 0) return;
  const WaitCtx wait{&abort_flag, c.status};
  const int bytes_kv = c.e4m3 ? c.d : 2 * c.d;  // of a token and head
  const int per_run = 2 * c.kv_pieces + c.exp_pieces, per_move = c.runs * per_run;
  const long long units = (long long)count * per_move, stride = (long long)gridDim.x * kCopyWarps;
  const long long page_rows = (long long)c.Hkv * c.page_size;
  auto unit = [&](long long u) {
    Unit x{nullptr, nullptr, 0};
    if (u >= units) return x;
    const int move = (int)(u / per_move), rest = (int)(u - (long long)move * per_move);
    int src, dst;
    if constexpr (kMode == kDirect) {
      src = list[move];
      dst = list[kCopyDirect + move];
    } else {
      src = __ldcg(c.moves.src + move);
      dst = __ldcg(c.moves.dst + move);
    }
    if (src < 0) return x;
    const int run = rest / per_run, part = rest - run * per_run;
    const int which = part < c.kv_pieces ? 0 : part < 2 * c.kv_pieces ? 1 : 2;
    const int bytes = which == 2 ? 2 : bytes_kv;
    const long long tokens = c.moves.tokens ? (long long)__ldcg(c.moves.tokens + move) : page_rows;
    const long long at = (long long)(part - which * c.kv_pieces) * kPiece;
    const long long off = (long long)run * c.page_size * bytes + at, page = page_rows * bytes;
    const long long left = tokens * bytes - at;
    if (left <= 0) return x;
    x.n = (int)imin64(left, kPiece);
    const void* from = which == 0 ? c.from[0] : which == 1 ? c.from[1] : c.from[2];
    void* to = which == 0 ? c.to[0] : which == 1 ? c.to[1] : c.to[2];
    x.from = static_cast<const uint8_t*>(from) + src * page + off;
    x.to = static_cast<uint8_t*>(to) + dst * page + off;
    return x;
  };
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
    const Unit mine = unit(u + lane * stride);
#pragma unroll 1
    for (uint32_t todo = __ballot_sync(0xffffffffu, mine.n > 0); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1, n = __shfl_sync(0xffffffffu, mine.n, who), whole = n & ~15;
      const uint8_t* from = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.from), who));
      uint8_t* to = reinterpret_cast<uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.to), who));
      if (lane < (n - whole) / 2)
        reinterpret_cast<uint16_t*>(to + whole)[lane] = reinterpret_cast<const uint16_t*>(from + whole)[lane];
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
cudaError_t launch(const PageCopy& c, const CompactArgs& compact, const CopyPlanArgs& plan, long long most,
                   int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem((const void*)page_copy_kernel<kMode>, kCopySmem, done);
  if (e != cudaSuccess) return e;
  const long long units = most * c.runs * (2 * c.kv_pieces + c.exp_pieces);
  const long long ctas = imin64((units + kCopyWarps - 1) / kCopyWarps, num_sms > 0 ? num_sms : 1);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ctas > 0 ? ctas : 1));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = kCopySmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kMode == kDirect ? 0 : 1;  // the others follow a plan kernel
  return cudaLaunchKernelEx(&cfg, page_copy_kernel<kMode>, c, compact, plan);
}

// Runs and pieces of a move: whole pages, or their first tokens.
PageCopy with_pieces(const PageCopy& copy) {
  PageCopy c = copy;
  c.runs = c.moves.tokens ? c.Hkv : 1;
  const long long tokens = c.moves.tokens ? c.page_size : (long long)c.Hkv * c.page_size;
  c.kv_pieces = (int)((tokens * (c.e4m3 ? c.d : 2 * c.d) + kPiece - 1) / kPiece);
  c.exp_pieces = c.e4m3 ? (int)((tokens * 2 + kPiece - 1) / kPiece) : 0;
  return c;
}

}  // namespace

cudaError_t launch_page_copy(const PageCopy& c, int num_sms, cudaStream_t st) {
  return launch<kListed>(with_pieces(c), CompactArgs{}, CopyPlanArgs{}, c.moves.most, num_sms, st);
}
cudaError_t launch_compact_copy(const PageCopy& c, const CompactArgs& compact, int num_sms, cudaStream_t st) {
  // (the CTAs rewrite the table's rows too)
  return launch<kCompact>(with_pieces(c), compact, CopyPlanArgs{}, (long long)c.moves.most + compact.s.B, num_sms, st);
}
cudaError_t launch_direct_copy(const PageCopy& c, const CopyPlanArgs& plan, int num_sms, cudaStream_t st) {
  return launch<kDirect>(with_pieces(c), CompactArgs{}, plan, plan.n, num_sms, st);
}

}  // namespace attn
