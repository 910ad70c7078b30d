// The paged cache as the kernels see it: one problem description shared by the cache
// writer and reader, the chunk attention and the e4m3 decode, and the device functions
// that find a packed row's sequence, position and cache slot.
#pragma once

#include "paged.h"
#include "paged_index.cuh"
#include "ptx.cuh"

namespace attn {

constexpr float kPagedLog2e = 1.4426950408889634f;
constexpr float kPagedLn2 = 0.69314718055994531f;

// The merge of the key chunks is launched as a programmatic dependent of the attention kernel:
// its CTAs may start once every CTA of that kernel has called grid_dependents_launch (or
// ended), and read its results only after grid_dependency_wait, which returns when it has
// completed. Against an ordinary launch: 2 us less per call (two sequences of 131072: 113.8 ->
// 111.7 us with a flushed L2).
__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// 2-D tiled load of one box.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// Maximum that keeps a NaN (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The new tokens of a sequence (nothing when its device inputs cannot be followed).
struct Span {
  int row0;  // packed row of the first new token
  int n;     // new tokens
  int L;     // cached tokens, the new ones included
};

__device__ __forceinline__ bool span_ok(const PagedProblem& p, int o0, int o1, int L) {
  return paged_span_ok(p.T, p.max_new, p.max_seq_len, o0, o1, L);
}

// Without offsets (decode) every sequence has p.max_new new tokens.
__device__ __forceinline__ Span load_span(const PagedProblem& p, int b) {
  const int o0 = p.offsets ? __ldg(p.offsets + b) : b * p.max_new;
  const int o1 = p.offsets ? __ldg(p.offsets + b + 1) : o0 + p.max_new;
  const int L = __ldg(p.seq_lens + b);
  if (!span_ok(p, o0, o1, L)) return Span{0, 0, 0};
  return Span{o0, o1 - o0, L};
}

// Reports every sequence whose inputs break the rules, once per launch (called by one CTA).
__device__ __forceinline__ void report_bad_spans(const PagedProblem& p) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int o0 = p.offsets ? __ldg(p.offsets + b) : b * p.max_new;
    const int o1 = p.offsets ? __ldg(p.offsets + b + 1) : o0 + p.max_new;
    if (!span_ok(p, o0, o1, __ldg(p.seq_lens + b)) || (b == 0 && o0 != 0))
      atomicOr(p.status, DEV_BAD_INPUT);
  }
}

// Sequence that holds packed row t, by a 32-way search of the offsets (all lanes together):
// the last b with offsets[b] <= t. One or two dependent loads up to B = 1024, where a
// binary search needs ten.
__device__ __forceinline__ int find_sequence(const PagedProblem& p, int t, int lane) {
  if (!p.offsets) return t / p.max_new;
  int lo = 0, len = p.B;  // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const bool le = at < len && __ldg(p.offsets + lo + at) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    lo += k * step;
    len = imin(step, len - k * step);
  }
  return lo;
}

// Cache row of a token of sequence b (see paged_row). pos must lie inside the page table.
__device__ __forceinline__ long long cache_row(const PagedProblem& p, int b, int pos, int head) {
  const int at = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
  const int page = __ldg(p.page_table + (size_t)b * p.max_pages + at);
  return paged_row(page, p.num_pages, p.Hkv, p.page_size, head, pos - at * p.page_size);
}

// 2^(byte - 127) as a float; byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float exp_byte_scale(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Two e4m3 codes (the low 16 bits of w) to a half2 word; every e4m3 value is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)w));
  return r;
}
// Four e4m3 codes to two half2 words.
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

}  // namespace attn
