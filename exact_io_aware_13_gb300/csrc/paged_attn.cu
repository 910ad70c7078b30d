// Attention of packed rows over the paged cache, one warp per row on the CUDA cores: the
// plain form of the recurrence ("FlashAttention/es", "El truco del softmax en línea").
#include "paged.cuh"
#include "paged_out.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;

// Lane l holds columns l * D / 32 .. of q, of each key and value, and of O.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) paged_row_kernel(const PagedAttention a) {
  constexpr int kC = D / 32;
  const PagedProblem& p = a.p;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) report_bad_spans(p);
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / a.Hq), h = (int)(unit % a.Hq);
  if (t >= p.T) return;
  const int b = find_sequence(p, t, lane);
  const Span s = load_span(p, b);
  const int i = t - s.row0;
  if (i < 0 || i >= s.n) return;
  const long long ti = p.offsets ? t : i, bi = p.offsets ? 0 : b;
  int lo, hi;
  decode_row_keys(a.mask_kind, a.window, s.L, s.n, i, lo, hi);
  const int pos = s.L - s.n + i;
  const __nv_bfloat16* q = a.q + bi * a.q_batch + ti * a.q_token + h * a.q_head + lane * kC;
  float qv[kC], acc[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    qv[c] = __bfloat162float(q[c]);
    acc[c] = 0.f;
  }
  const float slope = (a.score_kind & ATTN_SCORE_ALIBI) ? alibi_slope(h, a.Hq) : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    const long long row = cache_row(p, b, j, h / a.G);
    if (row < 0) {
      if (lane == 0) atomicOr(p.status, DEV_BAD_INPUT);
      continue;
    }
    float kv[kC], vv[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const long long e = row * D + lane * kC + c;
      if constexpr (kE4m3) {
        kv[c] = f16x2_to_float2(e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.k_cache)[e])).x *
                exp_byte_scale(p.kv_exp[row * 2]);
        vv[c] = f16x2_to_float2(e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.v_cache)[e])).x *
                exp_byte_scale(p.kv_exp[row * 2 + 1]);
      } else {
        kv[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.k_cache)[e]);
        vv[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[e]);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) x = fmaf(qv[c], kv[c], x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x = x * a.scale - slope * (float)(pos - j);
    if (a.score_kind & ATTN_SCORE_SOFTCAP) x = a.softcap * tanhf(x / a.softcap);
    const float m_new = fmaxf(m, x);
    const float corr = m_new == -INFINITY ? 1.f : expf(m - m_new);
    const float w = m_new == -INFINITY ? 0.f : expf(x - m_new);
    l = l * corr + w;
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = acc[c] * corr + w * vv[c];
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* o = a.o + bi * a.o_batch + ti * a.o_token + h * a.o_head + lane * kC;
#pragma unroll
  for (int c = 0; c < kC; ++c) o[c] = __float2bfloat16(acc[c] * inv);
  if (lane == 0)
    a.lse[bi * a.l_batch + ti * a.l_token + h * a.l_head] = l > 0.f ? m + logf(l) : -INFINITY;
}

// Merge of the key chunks' partial results, one warp per row, in chunk order:
//   M = max_c L2_c, w_c = 2^(L2_c - M), O = sum_c w_c O_c / sum_c w_c, L = M + log2 sum_c w_c.
// Only chunks that hold keys of the row were written.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged_merge_kernel(const PagedAttention a) {
  constexpr int kC = D / 32;
  const PagedProblem& p = a.p;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / a.Hq), h = (int)(unit % a.Hq);
  if (t >= p.T) return;
  const int b = find_sequence(p, t, lane);
  const Span s = load_span(p, b);
  const int i = t - s.row0;
  if (i < 0 || i >= s.n) return;
  int lo, hi;
  decode_row_keys(a.mask_kind, a.window, s.L, s.n, i, lo, hi);
  const int ca = hi > lo ? lo / a.chunk : 0, cb = hi > lo ? (hi - 1) / a.chunk + 1 : 0;
  const long long rows = (long long)p.T * a.Hq, row = (long long)t * a.Hq + h;
  float M = -INFINITY;
  for (int c = ca + lane; c < cb; c += 32) M = fmaxf(M, a.part_lse[c * rows + row]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float W = 0.f, acc[kC];
#pragma unroll
  for (int e = 0; e < kC; ++e) acc[e] = 0.f;
  if (M > -INFINITY)
    for (int c = ca; c < cb; ++c) {
      const float w = ex2_approx(a.part_lse[c * rows + row] - M);
      W += w;
      const float* src = a.part_o + (c * rows + row) * D + lane * kC;
#pragma unroll
      for (int e = 0; e < kC; ++e) acc[e] = fmaf(w, src[e], acc[e]);
    }
  const float inv = W > 0.f ? 1.f / W : 0.f;
#pragma unroll
  for (int e = 0; e < kC; ++e) acc[e] *= inv;
  PagedAttention out = a;
  out.n_chunks = 1;
  store_row<D>(out, b, t, i, h, 0, lane, acc, W > 0.f ? M + log2f(W) : -INFINITY);
}

cudaError_t launch_merge(const PagedAttention& a, cudaStream_t st) {
  const long long blocks = ((long long)a.p.T * a.Hq + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.p.d == 64) paged_merge_kernel<64><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
  else paged_merge_kernel<128><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttention& a, const PagedMaps& maps,
                                   cudaStream_t st) {
  const long long rows = (long long)a.p.T * a.Hq;
  if (rows == 0) return cudaSuccess;
  if (paged_few_rows(a)) {
    const cudaError_t e = launch_paged_rows(a, maps, st);
    return e != cudaSuccess || a.n_chunks == 1 ? e : launch_merge(a, st);
  }
  const long long blocks = (rows + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)blocks, t = kWarps * 32;
  const bool e = a.p.kv_exp != nullptr;
  if (a.p.d == 64) e ? paged_row_kernel<64, true><<<g, t, 0, st>>>(a) : paged_row_kernel<64, false><<<g, t, 0, st>>>(a);
  else e ? paged_row_kernel<128, true><<<g, t, 0, st>>>(a) : paged_row_kernel<128, false><<<g, t, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
