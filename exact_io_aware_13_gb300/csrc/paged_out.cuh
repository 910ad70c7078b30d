// Where a paged attention kernel puts a finished row: the output itself, or a partial
// result of one key chunk for the merge.
#pragma once

#include "paged.cuh"

namespace attn {

// One warp writes row (t, h) of sequence b (t: its packed row, i: its index among the new
// tokens): lane l holds columns l * D / 32 .. of O / l, l2 is the row's log2-sum-exp over
// key chunk cc.
template <int D>
__device__ __forceinline__ void store_row(const PagedAttention& a, int b, int t, int i, int h,
                                          int cc, int lane, const float (&v)[D / 32], float l2) {
  constexpr int kC = D / 32;
  if (a.n_chunks > 1) {
    const long long row = ((long long)cc * a.p.T + t) * a.Hq + h;
    float* dst = a.part_o + row * D + lane * kC;
    if constexpr (kC == 4) *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<float2*>(dst) = make_float2(v[0], v[1]);
    if (lane == 0) a.part_lse[row] = l2;
    return;
  }
  const long long ti = a.p.offsets ? t : i, bi = a.p.offsets ? 0 : b;
  __nv_bfloat16* dst = a.o + bi * a.o_batch + ti * a.o_token + h * a.o_head + lane * kC;
  if constexpr (kC == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(v[0], v[1]);
  if (lane == 0) a.lse[bi * a.l_batch + ti * a.l_token + h * a.l_head] = l2 * kPagedLn2;
}

}  // namespace attn
