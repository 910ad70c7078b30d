// Attention of packed rows over the paged cache: the choice of kernel, and the merge of the
// key chunks' partial results.
#include "paged.cuh"
#include "paged_out.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;

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
    for (int c0 = ca; c0 < cb; c0 += 4) {  // four chunks' loads in flight
      float l2[4], v[4][kC];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool in = c0 + k < cb;
        const long long at = imin(c0 + k, cb - 1) * rows + row;
        l2[k] = in ? a.part_lse[at] : -INFINITY;
        const float* src = a.part_o + at * D + lane * kC;
        if constexpr (kC == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[k][0] = f.x; v[k][1] = f.y; v[k][2] = f.z; v[k][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          v[k][0] = f.x; v[k][1] = f.y;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = ex2_approx(l2[k] - M);
        W += w;
#pragma unroll
        for (int e = 0; e < kC; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
      }
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
  const cudaError_t e = a.p.kv_exp ? launch_paged_tiles_e4m3(a, st) : launch_paged_tiles_bf16(a, maps, st);
  return e != cudaSuccess || a.n_chunks == 1 ? e : launch_merge(a, st);
}

}  // namespace attn
