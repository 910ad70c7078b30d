// Attention of packed rows over the paged cache: the choice of kernel, and the merge of the
// key chunks' partial results.
#include "paged.cuh"
#include "paged_out.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;

// Merge of the key chunks' partial results, in a fixed order:
//   M = max_c L2_c, W = sum_c 2^(L2_c - M), O = sum_c (2^(L2_c - M) / W) O_c, L = M + log2 W.
// The weights are divided before they meet the values, which may lie near the top of fp32's
// range. Only chunks that hold keys of the row were written. A row takes one warp, or with many
// chunks and few rows eight (each a contiguous part of them, joined through shared memory):
// a lone warp's loads for 98 chunks of a 131072-token sequence took 25 us one after the other.
template <int D, int kPerRow>
__global__ void __launch_bounds__(kWarps * 32) paged_merge_kernel(const PagedAttention a) {
  constexpr int kC = D / 32;
  __shared__ float sm[kPerRow > 1 ? kWarps : 1][D + 4];
  const PagedProblem& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % kPerRow;
  const long long unit = ((long long)blockIdx.x * kWarps + warp) / kPerRow;
  const int t = (int)(unit / a.Hq), h = (int)(unit % a.Hq);
  const int b = find_sequence(p, imin(t, p.T - 1), lane);
  const Span s = load_span(p, b);
  // Launched while the attention kernel's last CTAs write their results: everything above
  // reads inputs only; no thread passes (or leaves) before that kernel has completed.
  grid_dependency_wait();
  if (t >= p.T) return;  // (with eight warps per row a CTA has one row)
  const int i = t - s.row0;
  if (i < 0 || i >= s.n) return;
  int lo, hi;
  decode_row_keys(a.mask_kind, a.window, s.L, s.n, i, lo, hi);
  const int ca = hi > lo ? lo / a.chunk : 0, cb = hi > lo ? (hi - 1) / a.chunk + 1 : 0;
  const int each = (cb - ca + kPerRow - 1) / kPerRow;
  const int c_begin = imin(ca + part * each, cb), c_end = imin(c_begin + each, cb);
  const long long rows = (long long)p.T * a.Hq, row = (long long)t * a.Hq + h;
  const int c_lane = c_begin + lane;
  const float first = c_lane < c_end ? a.part_lse[c_lane * rows + row] : -INFINITY;
  float M = first;
  for (int c = c_lane + 32; c < c_end; c += 32) M = max_nan(M, a.part_lse[c * rows + row]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
  float W = 0.f, acc[kC];
#pragma unroll
  for (int e = 0; e < kC; ++e) acc[e] = 0.f;
  if (M != -INFINITY) {  // (a NaN chunk makes the row NaN)
    W = ex2_approx(first - M);
    for (int c = c_lane + 32; c < c_end; c += 32) W += ex2_approx(a.part_lse[c * rows + row] - M);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) W += __shfl_xor_sync(0xffffffffu, W, off);
    const float inv = 1.f / W;  // W >= 1
    for (int c0 = c_begin; c0 < c_end; c0 += 4) {  // four chunks' loads in flight
      float l2[4], v[4][kC];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long long at = imin(c0 + k, c_end - 1) * rows + row;
        l2[k] = c0 + k < c_end ? a.part_lse[at] : -INFINITY;
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
        const float w = ex2_approx(l2[k] - M) * inv;
#pragma unroll
        for (int e = 0; e < kC; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
      }
    }
  }
  if constexpr (kPerRow > 1) {
#pragma unroll
    for (int e = 0; e < kC; ++e) sm[warp][lane * kC + e] = acc[e];
    if (lane == 0) {
      sm[warp][D] = M;
      sm[warp][D + 1] = W;
    }
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int k = 0; k < kPerRow; ++k) M = max_nan(M, sm[k][D]);
    float share[kPerRow];
    W = 0.f;
#pragma unroll
    for (int k = 0; k < kPerRow; ++k) {
      share[k] = sm[k][D] == -INFINITY ? 0.f : ex2_approx(sm[k][D] - M) * sm[k][D + 1];
      W += share[k];
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
#pragma unroll
    for (int e = 0; e < kC; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kPerRow; ++k)
#pragma unroll
      for (int e = 0; e < kC; ++e) acc[e] = fmaf(share[k] * inv, sm[k][lane * kC + e], acc[e]);
  }
  PagedAttention out = a;
  out.n_chunks = 1;
  store_row<D>(out, b, t, i, h, 0, lane, acc, W == 0.f ? -INFINITY : M + log2f(W));
}

template <int D, int kPerRow>
cudaError_t launch_merge_as(const PagedAttention& a, cudaStream_t st) {
  const long long blocks = ((long long)a.p.T * a.Hq * kPerRow + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, kPerRow>, a);
}
cudaError_t launch_merge(const PagedAttention& a, cudaStream_t st) {
  // Eight warps per row once a lone warp would take more than two turns of its four loads, as
  // long as the rows are few: from some 2000 rows on, one warp each keeps enough loads in flight
  // and needs no join. The kernel alone, one warp | eight (d = 128): 13 chunks, 64 rows 8.0 | 4.5
  // us, 1024 8.6 | 8.3, 4096 10.8 | 19.6, 16384 26 | 64; 102 chunks, 64 rows 37 | 8.5, 1024
  // 37 | 17, 4096 44 | 48, 16384 143 | 166.
  if (a.n_chunks > 8 && (long long)a.p.T * a.Hq <= 2048)
    return a.p.d == 64 ? launch_merge_as<64, 8>(a, st) : launch_merge_as<128, 8>(a, st);
  return a.p.d == 64 ? launch_merge_as<64, 1>(a, st) : launch_merge_as<128, 1>(a, st);
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
  const cudaError_t e = a.p.e4m3 ? launch_paged_tiles_e4m3(a, st) : launch_paged_tiles_bf16(a, maps, st);
  return e != cudaSuccess || a.n_chunks == 1 ? e : launch_merge(a, st);
}

}  // namespace attn
