// Device pieces of the pool's plan kernels. A plan is integer work over a few hundred KB that
// needs several grid-wide steps, so each runs as one thread-block cluster: its barrier orders
// global memory between the CTAs, and counts are exchanged through distributed shared memory.
#pragma once

#include "pool.h"
#include "ptx.cuh"

namespace attn {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// A peer's shared memory may be written once its CTA has started: every thread arrives early
// and waits before the first such write.
__device__ __forceinline__ void cluster_started_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_started_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// Every thread of the cluster; memory written before is visible after it, in every CTA.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Writes v into the same shared-memory word of CTA `cta` of this cluster.
__device__ __forceinline__ void store_peer(const void* word, uint32_t cta, unsigned long long v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(word)), "r"(cta));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// One total per CTA, known to all of them after the next cluster_sync.
struct Totals {
  unsigned long long of[kPlanMaxCtas];
  // by one warp of every CTA, the same v in all its lanes
  __device__ __forceinline__ void publish(unsigned long long v, int lane) {
    if (lane < (int)cluster_size()) store_peer(&of[cluster_rank()], lane, v);
  }
  __device__ __forceinline__ unsigned long long sum() const { return before(cluster_size()); }
  __device__ __forceinline__ unsigned long long before(uint32_t cta) const {
    unsigned long long t = 0;
    for (uint32_t c = 0; c < cta; ++c) t += of[c];
    return t;
  }
};

__device__ __forceinline__ int pages_of(const PoolState& s, int tokens) {
  return s.page_shift >= 0 ? (int)(((unsigned)tokens + s.page_size - 1) >> s.page_shift)
                           : (int)(((unsigned)tokens + s.page_size - 1) / s.page_size);
}
__device__ __forceinline__ int page_index(const PoolState& s, int token) {
  return s.page_shift >= 0 ? token >> s.page_shift : token / s.page_size;
}
__device__ __forceinline__ bool length_ok(const PoolState& s, int L) {
  return L >= 0 && (long long)L <= (long long)s.max_pages * s.page_size;
}

// Contiguous shares: CTA c of n gets [lo, hi) of `total`.
struct Share {
  int lo, hi;
  __device__ __forceinline__ Share(int total, uint32_t c, uint32_t n) {
    const long long per = ((long long)total + n - 1) / n;
    lo = (int)(per * c < total ? per * c : total);
    hi = (int)(per * (c + 1) < total ? per * (c + 1) : total);
  }
};

// Exclusive prefix of v over the CTA's threads; `total` is the CTA's sum. warp_sums: shared
// memory of kPlanWarps words, free again after the call's second barrier.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* warp_sums,
                                                         unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  unsigned long long w = warp_sums[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const unsigned long long base = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return x - v + (warp > 0 ? base : 0);
}

}  // namespace attn
