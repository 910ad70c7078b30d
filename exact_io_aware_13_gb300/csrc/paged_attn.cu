// Attention of packed rows over the paged cache, one warp per row on the CUDA cores: the
// plain form of the recurrence ("FlashAttention/es", "El truco del softmax en línea").
#include "paged.cuh"

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

}  // namespace

cudaError_t launch_paged_attention(const PagedAttention& a, int num_sms, cudaStream_t st) {
  (void)num_sms;
  const long long rows = (long long)a.p.T * a.Hq;
  if (rows == 0) return cudaSuccess;
  const long long blocks = (rows + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)blocks, t = kWarps * 32;
  const bool e = a.p.kv_exp != nullptr;
  if (a.p.d == 64) e ? paged_row_kernel<64, true><<<g, t, 0, st>>>(a) : paged_row_kernel<64, false><<<g, t, 0, st>>>(a);
  else e ? paged_row_kernel<128, true><<<g, t, 0, st>>>(a) : paged_row_kernel<128, false><<<g, t, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
