// Verification of drafted tokens against a target model's probabilities, from given random
// numbers. Draft i of a sequence stays iff u_i q_i(x_i) < p_i(x_i) (the products of fp32 values
// are exact in fp64); with a the first that does not, the next token is drawn from
// max(p_a - q_a, 0), else from the last row of p: the lowest x with cumsum(w)(x) > u * sum(w).
//
// One thread-block cluster per sequence, each warp a contiguous piece of the vocabulary. Sums
// have to be so exact that the drawn token does not depend on their order: weights are p - q
// and its rounding error, accumulated as pairs of fp32 (about 48 bits), since fp64 runs at a
// sixty-fourth of the fp32 rate. HBM-bound: V values of p, and of q, per sequence.
#include <cuda_fp16.h>

#include "paged.cuh"
#include "pool.cuh"

namespace attn {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// An unevaluated sum of two fp32 numbers.
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float err) {
    const float s = hi + x, t = s - hi;  // Knuth's two-sum
    lo += ((hi - (s - t)) + (x - t)) + err;
    hi = s;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// A weight max(p - q, 0) and its rounding error (exact: p >= q >= 0). What is not a positive
// finite number counts as no weight.
struct Weight {
  float w, err;
  __device__ __forceinline__ Weight(float p, float q) {
    w = p - q;
    err = (p - w) - q;
    if (!(w > 0.f && w < INFINITY)) w = err = 0.f;
  }
};

// The p and q of one row, in groups of kVec elements that start at 16-byte boundaries of p.
// Elements outside [0, V) and skipped ones have no weight.
template <class T>
struct RowReader {
  static constexpr int kVec = 16 / sizeof(T);
  const T *p, *q;
  int V, shift, skip;  // element of group g, lane j: g * kVec + j - shift; skip: weightless token
  bool q_vec;          // q's groups start at 16-byte boundaries too
  __device__ __forceinline__ RowReader(const T* p_, const T* q_, int V_, int skip_)
      : p(p_), q(q_), V(V_), skip(skip_) {
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    q_vec = q && ((reinterpret_cast<uintptr_t>(q) & 15) / sizeof(T)) == (uintptr_t)shift;
  }
  __device__ __forceinline__ int groups() const { return (int)(((long long)V + shift + kVec - 1) / kVec); }
  __device__ __forceinline__ int first(int g) const { return g * kVec - shift; }
  __device__ __forceinline__ void load(int g, float (&pv)[kVec], float (&qv)[kVec]) const {
    const int v0 = first(g);
    if (v0 >= 0 && v0 + kVec <= V) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p + v0));
      const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
      for (int j = 0; j < kVec; ++j) pv[j] = to_float(e[j]);
      if (q_vec) {
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(q + v0));
        const T* f = reinterpret_cast<const T*>(&y);
#pragma unroll
        for (int j = 0; j < kVec; ++j) qv[j] = to_float(f[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) qv[j] = q ? to_float(q[v0 + j]) : 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const bool in = v0 + j >= 0 && v0 + j < V;
        pv[j] = in ? to_float(p[v0 + j]) : 0.f;
        qv[j] = in && q ? to_float(q[v0 + j]) : 0.f;
      }
    }
    if (skip >= v0 && skip < v0 + kVec) {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (v0 + j == skip) pv[j] = 0.f;
    }
  }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// First part of `n` whose running sum passes `threshold` (or the last with a sum at all, -1
// without one); `before` is the sum in front of it. Every caller sees the same numbers.
__device__ __forceinline__ int pick_part(const double* sums, int n, double base, double threshold,
                                         double& before) {
  int last = -1;
  before = base;
  double run = base;
  for (int i = 0; i < n; ++i) {
    if (!(sums[i] > 0.0)) continue;
    last = i;
    before = run;
    run += sums[i];
    if (run > threshold) break;
  }
  return last;
}

// The token of a warp's groups [g0, g1) at which the running sum from `base` passes `threshold`;
// the last with any weight if none does.
template <class T>
__device__ int find_token(const RowReader<T>& row, int g0, int g1, double base, double threshold, int lane) {
  constexpr int kVec = RowReader<T>::kVec;
  int last = -1;
  for (int g = g0; g < g1; g += 32) {
    float pv[kVec], qv[kVec];
    const bool in = g + lane < g1;
    if (in) row.load(g + lane, pv, qv);
    double mine = 0.0;
    int mine_last = -1;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (!in) continue;
      const Weight w(pv[j], qv[j]);
      mine += (double)w.w + (double)w.err;
      if (w.w > 0.f) mine_last = row.first(g + lane) + j;
    }
    double run = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, base + run > threshold && mine > 0.0);
    if (over) {
      const int who = __ffs(over) - 1;
      int token = -1;
      if (lane == who) {
        double c = base + (run - mine);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const Weight w(pv[j], qv[j]);
          c += (double)w.w + (double)w.err;
          if (w.w > 0.f && c > threshold && token < 0) token = row.first(g + lane) + j;
        }
        if (token < 0) token = mine_last;
      }
      return __shfl_sync(0xffffffffu, token, who);
    }
    base += __shfl_sync(0xffffffffu, run, 31);
    const uint32_t some = __ballot_sync(0xffffffffu, mine_last >= 0);
    if (some) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(some));
  }
  return last;
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a) {
  __shared__ int s_kept;
  __shared__ double warp_sums[kVerifyWarps];
  __shared__ Totals sums;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = cluster_rank(), ctas = cluster_size();
  const int b = blockIdx.x / ctas;
  const int r0 = __ldg(a.offsets + b), r1 = __ldg(a.offsets + b + 1);
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= a.T && (b > 0 || r0 == 0);
  const int n = ok ? r1 - r0 : 0;
  if (!ok && threadIdx.x == 0) atomicOr(a.status, DEV_BAD_INPUT);
  const T* target = static_cast<const T*>(a.target);
  const T* draft = static_cast<const T*>(a.draft);
  if (n == 0) {  // the same in every CTA of the cluster
    if (cta == 0 && threadIdx.x == 0) {
      a.accepted[b] = 0;
      a.next_tokens[b] = -1;
      if (a.kept_lens) a.kept_lens[b] = __ldg(a.seq_lens + b);
    }
    return;
  }
  cluster_started_arrive();
  if (warp == 0) {  // drafts that stay, 32 at a time
    int kept = n - 1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int t = r0 + i0 + lane;
      bool stays = true;
      if (i0 + lane < n - 1) {
        const int x = __ldg(a.tokens + t + 1);
        const double u = __ldg(a.accept_u + t);
        if (x >= 0 && x < a.V) {
          const double p = to_float(target[(size_t)t * a.target_stride + x]);
          const double q = draft ? to_float(draft[(size_t)t * a.draft_stride + x]) : 1.f;
          stays = u * q < p;
        } else {
          stays = false;
          atomicOr(a.status, DEV_BAD_INPUT);
        }
      }
      const uint32_t out = __ballot_sync(0xffffffffu, !stays);
      if (out) {
        kept = i0 + __ffs(out) - 1;
        break;
      }
    }
    if (lane == 0) s_kept = kept;
  }
  __syncthreads();
  cluster_started_wait();
  const int kept = s_kept, t = r0 + kept;
  const bool rejected = kept < n - 1;
  const T* p = target + (size_t)t * a.target_stride;
  const T* q = rejected && draft ? draft + (size_t)t * a.draft_stride : nullptr;
  const int skip = rejected && !draft ? __ldg(a.tokens + t + 1) : -1;
  // the warp's groups of a row shared by `warps` warps, and the sums of the CTA's warps over theirs
  int g0, g1;
  auto sum_row = [&](const RowReader<T>& row, int me, int warps) {
    constexpr int kVec = RowReader<T>::kVec;
    const int groups = row.groups(), per = ((groups + warps - 1) / warps + 31) / 32 * 32;
    g0 = (int)imin64((long long)me * per, groups);
    g1 = (int)imin64((long long)(me + 1) * per, groups);
    Pair sum;
    for (int g = g0 + lane; g < g1; g += 32) {
      float pv[kVec], qv[kVec];
      row.load(g, pv, qv);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const Weight w(pv[j], qv[j]);
        sum.add(w.w, w.err);
      }
    }
    const double mine = warp_sum(sum.value());
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    double x = 0.0;
    for (int w = 0; w < kVerifyWarps; ++w) x += warp_sums[w];
    return x;
  };
  const double u = __ldg(a.sample_u + b);
  auto draw = [&](const RowReader<T>& row, double before, double threshold) {
    double mine_before;
    if (pick_part(warp_sums, kVerifyWarps, before, threshold, mine_before) != warp) return;
    const int token = find_token(row, g0, g1, mine_before, threshold, lane);
    if (lane == 0) a.next_tokens[b] = token;
  };
  const RowReader<T> row(p, q, a.V, skip);
  const double mine = sum_row(row, cta * kVerifyWarps + warp, ctas * kVerifyWarps);
  if (warp == 0) sums.publish(__double_as_longlong(mine), lane);
  cluster_sync();
  double of[kPlanMaxCtas], total = 0.0;
  for (int c = 0; c < kPlanMaxCtas; ++c) {
    of[c] = c < (int)ctas ? __longlong_as_double(sums.of[c]) : 0.0;
    total += of[c];
  }
  if (total > 0.0) {
    double before;
    if (pick_part(of, ctas, 0.0, u * total, before) == (int)cta) draw(row, before, u * total);
  } else if (cta == 0) {
    // p <= q everywhere: from p itself, by one CTA (p = q, or rows without a weight: rare)
    const RowReader<T> all(p, nullptr, a.V, -1);
    total = rejected ? sum_row(all, warp, kVerifyWarps) : 0.0;
    if (total > 0.0) {
      draw(all, 0.0, u * total);
    } else if (threadIdx.x == 0) {
      a.next_tokens[b] = -1;
      atomicOr(a.status, DEV_BAD_INPUT);
    }
  }
  if (cta == 0 && threadIdx.x == 0) {
    a.accepted[b] = kept;
    if (a.kept_lens) a.kept_lens[b] = __ldg(a.seq_lens + b) - (n - 1 - kept);
  }
}

template <class T>
cudaError_t launch(const VerifyArgs& a, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.B * ctas);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t st) {
  const int ctas = a.V > 8192 ? 8 : 1;
  switch (a.type) {
    case ATTN_PROB_FP32: return launch<float>(a, ctas, st);
    case ATTN_PROB_BF16: return launch<__nv_bfloat16>(a, ctas, st);
    default: return launch<__half>(a, ctas, st);
  }
}

}  // namespace attn
