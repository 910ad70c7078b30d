// Verification of drafted tokens against a target model's probabilities, from given random
// numbers. Draft i of a sequence stays iff u_i q_i(x_i) < p_i(x_i) (the products of fp32 values
// are exact in fp64); with a the first that does not, the next token is drawn from
// max(p_a - q_a, 0), else from the last row of p: the lowest x with cumsum(w)(x) > u * sum(w).
//
// One thread-block cluster per sequence, each warp a contiguous piece of the vocabulary. Sums
// have to be so exact that the drawn token does not depend on their order: weights are p - q
// and its rounding error, accumulated as pairs of fp32 (two-sums whose errors add up apart: at most
// 2 n (n + 1) 2^-48 of a sum of n weights is lost, and n is at most 128 for rows of up to 2^20), since
// fp64 runs at a sixty-fourth of the fp32 rate: with fp64 sums over the warps and CTAs alone 128 sequences of
// 128000 bf16 tokens took 90 us. HBM-bound for a batch: V values of p, and of q, per sequence;
// for few sequences the chain offsets -> tokens -> p, q of the drafts -> rows -> token. Measured:
// 128 sequences of 8 drafts over 128000 bf16 tokens 21.5 us (61 MB, 12 us of it the stream), 200 over
// 50257 fp16 tokens without q 12.2 us, one over 32000 fp32 tokens 6.1 us, 585 over 256000 bf16
// tokens without drafts 64 us (4.7 TB/s).
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.cuh"
#include "pool.cuh"

namespace attn {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
// Pieces of a row whose sums are kept: of about 4096 tokens, which a CTA searches in 16 steps. One
// piece per warp for 585 sequences over 256000 tokens (32000 each) takes 93 us, of 4096 64 us.
constexpr int kMaxPieces = 256, kPieceTokens = 4096;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// An unevaluated sum of two fp32 numbers.
struct alignas(8) Pair {  // (one word of distributed shared memory)
  float hi, lo;
  __device__ __forceinline__ void add(float x, float err) {
    const float s = hi + x, t = s - hi;  // Knuth's two-sum
    lo += ((hi - (s - t)) + (x - t)) + err;
    hi = s;
  }
  __device__ __forceinline__ Pair normal() const {  // hi is the sum rounded
    Pair p;
    p.hi = hi + lo;
    p.lo = lo - (p.hi - hi);
    return p;
  }
};
__device__ __forceinline__ Pair operator+(Pair a, const Pair& b) {
  a.add(b.hi, b.lo);
  return a.normal();
}
__device__ __forceinline__ bool operator>(const Pair& a, const Pair& b) {  // both normal
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ Pair operator*(float u, const Pair& a) {
  Pair p;
  p.hi = u * a.hi;
  p.lo = fmaf(u, a.hi, -p.hi) + u * a.lo;
  return p.normal();
}
__device__ __forceinline__ bool some_weight(const Pair& p) { return p.hi > 0.f && p.hi < INFINITY; }
// u times the total weight, which a running sum has to pass. The product's low bits are held where
// it is at least 2^-76 (48 bits, and fp32 goes down to 2^-149). Below that both sides of every
// comparison are 2^96 times as large: exactly so, but for running sums that become infinite, which
// pass as they should, and for products below 2^-172, which every weight there is passes anyway.
struct Threshold {
  float scale;
  Pair at;
  __device__ __forceinline__ Threshold(float u, const Pair& total)
      : scale(u * total.hi < 0x1p-76f ? 0x1p96f : 1.f), at(u * scale * total) {}
  __device__ __forceinline__ bool passed(const Pair& run) const {  // normal
    return Pair{run.hi * scale, run.lo * scale} > at;
  }
};
// Two pairs, for the elements of even and of odd index.
struct Pair2 {
  uint64_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(uint64_t x) {
    const uint64_t s = add_f32x2(hi, x), t = sub_f32x2(s, hi);
    lo = add_f32x2(lo, add_f32x2(sub_f32x2(hi, sub_f32x2(s, t)), sub_f32x2(x, t)));
    hi = s;
  }
  __device__ __forceinline__ void add(uint64_t x, uint64_t err) {
    lo = add_f32x2(lo, err);
    add(x);
  }
  __device__ __forceinline__ Pair sum() const {
    Pair p, r;
    f32x2_split(hi, p.hi, r.hi);
    f32x2_split(lo, p.lo, r.lo);
    return p + r;
  }
};
__device__ __forceinline__ Pair shfl(const Pair& x, int lane) {
  return Pair{__shfl_sync(0xffffffffu, x.hi, lane), __shfl_sync(0xffffffffu, x.lo, lane)};
}

// The inclusive prefix of x over the warp's lanes.
__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, x.hi, off), __shfl_up_sync(0xffffffffu, x.lo, off)};
    if (lane >= off) x = y + x;
  }
  return x;
}

// First lane whose running sum passes the threshold, the last with a sum at all if none does.
// run: the inclusive prefix of mine. `before`: the running sum in front of that lane.
__device__ __forceinline__ int pick_lane(const Pair& mine, const Pair& run, const Threshold& threshold, int lane,
                                         Pair& before) {
  const uint32_t some = __ballot_sync(0xffffffffu, mine.hi > 0.f);
  const uint32_t over = some & __ballot_sync(0xffffffffu, threshold.passed(run));
  const int who = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
  const Pair x = shfl(run, who > 0 ? who - 1 : 0);
  before = who > 0 ? x : Pair{0.f, 0.f};
  return who;
}

// One row of p and, for a residual, of q; the weight of x is max(p - q, 0), none for `skip`. What
// is not a positive finite number counts as no weight. Vector loads take groups of kVec
// elements that start at 16-byte boundaries of p: group g holds g * kVec - shift onwards.
template <class T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T *p, *q;  // q may be null
  int V, skip, shift;
  // q's groups start at 16-byte boundaries too. If not, all elements go one by one (128 sequences of
  // 8 drafts over 50257 bf16 tokens 36 us, against 13): pad target and draft alike.
  bool vec;
  __device__ __forceinline__ Row(const T* p_, const T* q_, int V_, int skip_) : p(p_), q(q_), V(V_), skip(skip_) {
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    vec = !q || ((reinterpret_cast<uintptr_t>(q) & 15) / sizeof(T)) == (uintptr_t)shift;
  }
  // The weight and its rounding error (exact, since p >= q >= 0).
  __device__ __forceinline__ Pair weight(int x) const {
    const float a = to_float(p[x]), b = q ? to_float(q[x]) : 0.f;
    const float w = a - b, err = (a - w) - b;
    const bool ok = w > 0.f && w < INFINITY && x != skip;
    return Pair{ok ? w : 0.f, ok ? err : 0.f};
  }
  // Pieces of the row: whole steps of a warp's vector loads, from element at(i, per) on.
  __device__ __forceinline__ int per_piece(int pieces) const {
    const int groups = (int)(((unsigned)V + shift + kVec - 1) / kVec);
    return ((groups + pieces - 1) / pieces + 31) / 32 * 32 * kVec;
  }
  __device__ __forceinline__ int at(int i, int per) const {
    return (int)min(max((long long)per * i - shift, 0LL), (long long)V);
  }
  // Values 2j and 2j + 1 of a group.
  static __device__ __forceinline__ uint64_t two(const uint4& x, int j) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 4) {
      return f32x2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return f32x2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    } else {
      const float2 f = f16x2_to_float2(w[j]);
      return f32x2(f.x, f.y);
    }
  }
};

// A group without its element at byte `at`.
template <class T>
__device__ __forceinline__ uint4 cleared(const uint4& x, int at) {
  const uint32_t mask = sizeof(T) == 4 ? 0u : at & 2 ? 0x0000FFFFu : 0xFFFF0000u;
  uint4 r = x;
  if (at / 4 == 0) r.x &= mask;
  if (at / 4 == 1) r.y &= mask;
  if (at / 4 == 2) r.z &= mask;
  if (at / 4 == 3) r.w &= mask;
  return r;
}

// Sum over whole groups [g0, g1), a lane's share of them, two elements per instruction and kAhead
// groups in flight. What is no positive finite number spoils the sum for good, or sets `odd`,
// where it may not count (the residual max(p - q, 0) is p - min(p, q), whose rounding error needs
// no test then): the caller sees to that.
template <class T, bool kQ>
__device__ __forceinline__ Pair sum_groups(const Row<T>& row, int g0, int g1, int lane, bool& odd) {
  constexpr int kVec = Row<T>::kVec, kAhead = kQ ? 2 : 3;
  constexpr uint32_t kSigns = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
  const uint4* p = reinterpret_cast<const uint4*>(row.p - row.shift) + lane;
  const uint4* q = reinterpret_cast<const uint4*>(row.q - row.shift) + lane;
  const int skip_group = !kQ && row.skip >= 0 ? (row.skip + row.shift) / kVec - lane : -32;
  Pair2 sum;
  uint32_t bits = 0;
  auto add = [&](uint4 x, const uint4& y, int g) {
    if (!kQ) {
      if (g == skip_group) x = cleared<T>(x, (row.skip + row.shift) % kVec * (int)sizeof(T));
      bits |= x.x | x.y | x.z | x.w;
    }
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) {
      const uint64_t pv = Row<T>::two(x, j);
      if constexpr (kQ) {
        float pa, pb, qa, qb;
        f32x2_split(pv, pa, pb);
        f32x2_split(Row<T>::two(y, j), qa, qb);
        const uint64_t qv = f32x2(fminf(pa, qa), fminf(pb, qb)), w = sub_f32x2(pv, qv);
        sum.add(w, sub_f32x2(sub_f32x2(pv, w), qv));
      } else {
        sum.add(pv);
      }
    }
  };
  int g = g0;
#pragma unroll 1
  for (; g + 32 * kAhead <= g1; g += 32 * kAhead) {
    uint4 x[kAhead], y[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      x[i] = __ldg(p + g + 32 * i);
      if constexpr (kQ) y[i] = __ldg(q + g + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) add(x[i], y[i], g + 32 * i);
  }
#pragma unroll 1
  for (; g < g1; g += 32) {
    uint4 x = make_uint4(0, 0, 0, 0), y = x;  // (no weight)
    if (g + lane < g1) {
      x = __ldg(p + g);
      if constexpr (kQ) y = __ldg(q + g);
    }
    add(x, y, g);
  }
  odd = bits & kSigns;
  return sum.sum();
}

// Sum of the weights of [x0, x1), a piece of the row, by one warp; every lane has it.
template <class T, bool kQ>
__device__ __forceinline__ Pair sum_piece(const Row<T>& row, int x0, int x1, int lane) {
  constexpr int kVec = Row<T>::kVec;
  // whole groups [g0, g1), loaded as such; the elements beside them one by one
  const int shift = row.shift;
  int g0 = (x0 + shift + kVec - 1) / kVec, g1 = (int)(((long long)x1 + shift) / kVec);
  if (!row.vec || g1 < g0) g0 = g1 = (x1 + shift) / kVec;
  bool odd;
  Pair sum = sum_groups<T, kQ>(row, g0, g1, lane, odd);
  if (!__all_sync(0xffffffffu, sum.hi < INFINITY && !odd)) {
    g0 = g1 = (x1 + shift) / kVec;
    sum = Pair{0.f, 0.f};
  }
  const int lo = imin(imax(g0 * kVec - shift, x0), x1), hi = g1 > g0 ? g1 * kVec - shift : lo;
  const int left = lo - x0, single = left + (x1 - hi);
#pragma unroll 1
  for (int i = lane; i < single; i += 32) sum = sum + row.weight(i < left ? x0 + i : hi + (i - left));
  return shfl(warp_scan(sum, lane), 31);
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtasPerSm) verify_kernel(const VerifyArgs a) {
  __shared__ int s_kept;
  __shared__ Pair sums[kMaxPieces];  // of every piece of the row
  __shared__ Pair span_sums[kVerifyWarps];
  __shared__ int first_over, last_some;  // threads
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
#pragma unroll 1
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int t = r0 + i0 + lane;
      bool stays = true;
      if (i0 + lane < n - 1) {
        const int x = __ldg(a.tokens + t + 1);
        const float u = __ldg(a.accept_u + t);
        stays = x >= 0 && x < a.V;
        if (stays) {
          const float p = to_float(target[(size_t)t * a.target_stride + x]);
          const float q = draft ? to_float(draft[(size_t)t * a.draft_stride + x]) : 1.f;
          stays = (double)u * (double)q < (double)p && p > 0.f && p < INFINITY && fabsf(q) < INFINITY;  // exact
        } else {
          atomicOr(a.status, DEV_BAD_INPUT);
        }
      }
      const uint32_t out = __ballot_sync(0xffffffffu, !stays);
      if (out) {
        kept = i0 + __ffs(out) - 1;
        break;
      }
    }
    if (lane == 0) {
      s_kept = kept;
      first_over = kVerifyThreads;
      last_some = 0;
    }
  }
  __syncthreads();
  cluster_started_wait();
  const int kept = s_kept, t = r0 + kept;
  const bool rejected = kept < n - 1;
  const float u = __ldg(a.sample_u + b);
  if (cta == 0 && threadIdx.x == 0) {
    a.accepted[b] = kept;
    if (a.kept_lens) a.kept_lens[b] = __ldg(a.seq_lens + b) - (n - 1 - kept);
  }
  const int warps = ctas * kVerifyWarps, me = cta * kVerifyWarps + warp;
  // Pass 0: the residual, or the last row, by the whole cluster. Pass 1, where p <= q
  // everywhere (p = q): p itself, by one CTA.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const bool residual = rejected && pass == 0;
    const Row<T> row(target + (size_t)t * a.target_stride,
                     residual && draft ? draft + (size_t)t * a.draft_stride : nullptr, a.V,
                     residual && !draft ? __ldg(a.tokens + t + 1) : -1);
    // a warp's share in pieces small enough to be searched
    const int n_warps = pass == 0 ? warps : kVerifyWarps;
    const int each = imax(1, imin(kMaxPieces, a.V / kPieceTokens) / n_warps), pieces = n_warps * each;
    const int per = row.per_piece(pieces);
#pragma unroll 1
    for (int i = me * each; i < (me + 1) * each; ++i) {
      const Pair s = row.q ? sum_piece<T, true>(row, row.at(i, per), row.at(i + 1, per), lane)
                           : sum_piece<T, false>(row, row.at(i, per), row.at(i + 1, per), lane);
      if (pass > 0) {  // (its peers may be gone)
        if (lane == 0) sums[i] = s;
      } else if (lane < (int)ctas) {
        store_peer(&sums[i], lane, (unsigned long long)__float_as_uint(s.lo) << 32 | __float_as_uint(s.hi));
      }
    }
    if (pass == 0) cluster_sync();
    else __syncthreads();
    // every warp: the piece in which the running sum passes u times the total
    const int of_lane = (pieces + 31) / 32;
    Pair of{0.f, 0.f};
#pragma unroll 1
    for (int i = lane * of_lane; i < imin((lane + 1) * of_lane, pieces); ++i) of = of + sums[i];
    Pair run = warp_scan(of, lane), before;
    const Pair total = shfl(run, 31);
    if (!some_weight(total)) {
      if (cta != 0) return;
      if (total.hi == 0.f && residual) {
        __syncthreads();  // (sums has been read)
        continue;
      }
      if (threadIdx.x == 0) {  // no weight, or sums above fp32's range
        a.next_tokens[b] = -1;
        atomicOr(a.status, DEV_BAD_INPUT);
      }
      return;
    }
    const Threshold threshold(u, total);
    const int piece = pick_lane(of, run, threshold, lane, before) * of_lane;
    int last = piece;
    Pair base = before;
#pragma unroll 1
    for (int i = piece; i < imin(piece + of_lane, pieces); ++i) {  // among the lane's
      if (!(sums[i].hi > 0.f)) continue;
      last = i;
      base = before;
      before = before + sums[i];
      if (threshold.passed(before)) break;
    }
    if (pass == 0 && last / (kVerifyWarps * each) != (int)cta) return;
    // by the whole CTA: a contiguous span of the piece per thread, the running sums at its ends,
    // and the element where they enclose the threshold
    const int x0 = row.at(last, per), x1 = row.at(last + 1, per);
    const int span = (x1 - x0 + kVerifyThreads - 1) / kVerifyThreads;
    const int at = imin(x0 + (int)threadIdx.x * span, x1), end = imin(at + span, x1);
    Pair sum{0.f, 0.f};
#pragma unroll 4
    for (int x = at; x < end; ++x) {
      const Pair w = row.weight(x);
      sum.add(w.hi, w.lo);
    }
    sum = sum.normal();
    run = warp_scan(sum, lane);
    if (lane == 31) span_sums[warp] = run;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < warp; ++w) base = base + span_sums[w];
    run = base + run;
    before = Pair{__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
    if (lane == 0) before = base;
    if (sum.hi > 0.f) {
      if (threshold.passed(run)) atomicMin(&first_over, (int)threadIdx.x);
      else atomicMax(&last_some, (int)threadIdx.x);
    }
    __syncthreads();
    if ((int)threadIdx.x != (first_over < kVerifyThreads ? first_over : last_some)) return;
    int token = -1;
#pragma unroll 4
    for (int x = at; x < end; ++x) {
      const Pair w = row.weight(x);
      before.add(w.hi, w.lo);
      if (w.hi > 0.f) {
        token = x;
        if (threshold.passed(before.normal())) break;
      }
    }
    a.next_tokens[b] = token;
    return;
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
  static std::atomic<uint64_t> large[2];
  if (ctas > kPortableCtas && !large_clusters((const void*)verify_kernel<T>, cfg, large[0], large[1])) {
    cfg.gridDim = dim3((unsigned)a.B * kPortableCtas);
    attr[0].val.clusterDim.x = kPortableCtas;
  }
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int num_sms, cudaStream_t st) {
  const int ctas = verify_ctas(num_sms, a.B, a.V);
  switch (a.type) {
    case ATTN_PROB_FP32: return launch<float>(a, ctas, st);
    case ATTN_PROB_BF16: return launch<__nv_bfloat16>(a, ctas, st);
    default: return launch<__half>(a, ctas, st);
  }
}

}  // namespace attn
