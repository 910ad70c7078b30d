// Writing new tokens into the paged cache and reading them back.
//
// Writing to an e4m3 cache takes, per (token, kv head) and for K and V apart, the smallest
// power of two 2^e with amax <= 448 * 2^e and stores e4m3(x * 2^-e). With amax = m * 2^x,
// 1 <= m < 2, and 448 = 1.75 * 2^8, that is e = x - 8 for m <= 1.75, else x - 7. The scale
// is a power of two because a floating-point code loses nothing by it, and because
// code * 2^e is then exact in bf16 and in the attention kernels' fp16 operands.
//
// Both directions move each byte once: bound by HBM for long batches if the instructions per
// byte stay few, and by the chain of dependent loads (offsets, lengths, page table) for a
// decode step. A warp takes a packed row, or a slice of it, kChunksPerWarp 16-byte pieces at
// a time, all in flight at once; a row's first values are fetched before its slot is known.
// Measured (Hkv = 8, d = 128): 97000 tokens from e4m3 back to bf16 in 95 us = 6.3 TB/s;
// 29000 prompt tokens into e4m3 in 38 us = 4.6 TB/s (the quantiser's instructions).
#include "paged.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;          // warps per CTA, each with its own row slice
constexpr int kPieces = 4;         // bf16 pieces of 16 bytes per lane
constexpr int kChunksPerWarp = 32 * kPieces;

// Largest magnitude of 8 bf16 values, as bf16 bits (their order is the numbers'; infinities
// and NaN come out as 0x7F80 and above).
__device__ __forceinline__ uint32_t amax8(const uint4& w) {
  const uint32_t k = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
  return max(m & 0xFFFFu, m >> 16);
}
// The same over the finite values alone.
__device__ __forceinline__ uint32_t finite_amax8(const uint4& w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = u[i] & 0x7FFFu, hi = (u[i] >> 16) & 0x7FFFu;
    m = max(m, lo < 0x7F80u ? lo : 0u);
    m = max(m, hi < 0x7F80u ? hi : 0u);
  }
  return m;
}

// Biased exponent byte of the scale of a row whose largest magnitude has these bf16 bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax == 0) return 0;
  const int field = (int)(amax >> 7);  // x + 127; 0 for a subnormal, whose e is below -127
  const int e = (amax & 0x7Fu) <= 0x60u ? field - 8 : field - 7;
  return (uint32_t)(e < 0 ? 0 : e);
}

// Eight bf16 values times inv (a power of two) to eight e4m3 codes, lowest element first.
// (A value that is not finite has become NaN: an infinity would saturate to the largest
// finite code.)
__device__ __forceinline__ uint2 encode8(const uint4& w, float inv) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = pack_e4m3x2(__uint_as_float(u[i] << 16) * inv, __uint_as_float(u[i] & 0xFFFF0000u) * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ uint32_t nonfinite_to_nan(uint32_t u) {
  const uint32_t lo = (u & 0x7F80u) == 0x7F80u ? 0x7FC0u : u & 0xFFFFu;
  const uint32_t hi = (u & 0x7F800000u) == 0x7F800000u ? 0x7FC00000u : u & 0xFFFF0000u;
  return lo | hi;
}

struct CopyArgs {
  PagedProblem p;
  RowView in[2];            // write: K and V rows
  __nv_bfloat16* out[2];    // read: contiguous [T, Hkv, d]
  int slices;               // warps per row
  int per_warp;             // slices of kChunksPerWarp pieces that a warp takes, one by one
};

// The sequence and position of packed row t; false when it has none. A position outside the
// sequence is reported, not followed.
__device__ __forceinline__ bool locate(const PagedProblem& p, int t, int lane, int& b, int& pos) {
  b = find_sequence(p, t, lane);
  const Span s = load_span(p, b);
  const int i = t - s.row0;
  if (i < 0 || i >= s.n) return false;  // a row of no sequence, or bad inputs
  pos = s.L - s.n + i;
  if (pos < 0) {
    if (lane == 0) atomicOr(p.status, DEV_BAD_INPUT);
    return false;
  }
  return true;
}

// The 16-byte bf16 pieces of a warp's slice: lane l owns piece l % (D / 8) of (tensor, head)
// rows l / (D / 8), + 32 / (D / 8), ...; rows 0 .. Hkv - 1 are K heads, then come V heads.
template <int D>
struct Pieces {
  static constexpr int kPer = D / 8;
  int piece, row0, Hkv;
  __device__ __forceinline__ Pieces(int c0, int lane, int hkv)
      : piece(lane % kPer), row0((c0 + lane) / kPer), Hkv(hkv) {}
  __device__ __forceinline__ bool get(int j, int& head, bool& is_v) const {
    const int r = row0 + j * (32 / kPer);
    is_v = r >= Hkv;
    head = is_v ? r - Hkv : r;
    return r < 2 * Hkv;
  }
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) cache_write_kernel(const CopyArgs a) {
  constexpr int kPer = D / 8;  // lanes per (tensor, head) row: 8 or 16
  constexpr uint32_t kRow = kE4m3 ? D : 2 * D, kPiece = kRow / kPer;  // bytes in the cache
  const PagedProblem& p = a.p;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) report_bad_spans(p);
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long at = unit / a.slices;
  if (at >= p.T || at >= __ldg(p.offsets + p.B)) return;  // (the rows behind are not read)
  const int t = (int)at;
  int c0 = (int)(unit % a.slices) * a.per_warp * kChunksPerWarp;
  const int c_end = imin(c0 + a.per_warp * kChunksPerWarp, 2 * p.Hkv * kPer);
  const __nv_bfloat16* k = a.in[0].p + t * a.in[0].token_stride + lane % kPer * 8;
  const __nv_bfloat16* v = a.in[1].p + t * a.in[1].token_stride + lane % kPer * 8;
  auto load = [&](uint4 (&w)[kPieces]) {
    const Pieces<D> pieces(c0, lane, p.Hkv);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      int head;
      bool is_v;
      w[j] = make_uint4(0, 0, 0, 0);
      if (pieces.get(j, head, is_v))
        w[j] = __ldg(reinterpret_cast<const uint4*>(
            (is_v ? v : k) + head * (is_v ? a.in[1].head_stride : a.in[0].head_stride)));
    }
  };
  uint4 w[kPieces];
  load(w);  // on their way while the slot is looked up
  int b, pos;
  if (!locate(p, t, lane, b, pos)) return;
  const long long row0 = cache_row(p, b, pos, 0);
  if (row0 < 0) {
    if (lane == 0) atomicOr(p.status, DEV_BAD_INPUT);
    return;
  }
  uint8_t* kc = static_cast<uint8_t*>(p.k_cache) + row0 * kRow + lane % kPer * kPiece;
  uint8_t* vc = static_cast<uint8_t*>(p.v_cache) + row0 * kRow + lane % kPer * kPiece;
  uint8_t* ec = kE4m3 ? p.kv_exp + row0 * 2 : nullptr;
  for (;;) {
    const Pieces<D> pieces(c0, lane, p.Hkv);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      int head;
      bool is_v;
      const bool ok = pieces.get(j, head, is_v);
      const uint32_t down = (uint32_t)(head * p.page_size);  // cache rows from head 0's
      uint8_t* dst = (is_v ? vc : kc) + (size_t)down * kRow;
      if constexpr (!kE4m3) {
        if (ok) *reinterpret_cast<uint4*>(dst) = w[j];
      } else {
        uint32_t m = amax8(w[j]);  // the kPer lanes of one row agree on it
#pragma unroll
        for (int off = kPer / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
          m = finite_amax8(w[j]);
#pragma unroll
          for (int off = kPer / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
          w[j] = make_uint4(nonfinite_to_nan(w[j].x), nonfinite_to_nan(w[j].y), nonfinite_to_nan(w[j].z),
                            nonfinite_to_nan(w[j].w));
        }
        const uint32_t byte = scale_byte(m);
        const float inv = __uint_as_float((254u - byte) << 23);  // 2^-(byte - 127)
        if (ok) {
          *reinterpret_cast<uint2*>(dst) = encode8(w[j], inv);
          if (lane % kPer == 0) ec[down * 2ull + is_v] = (uint8_t)byte;
        }
      }
    }
    c0 += kChunksPerWarp;
    if (c0 >= c_end) return;
    load(w);
  }
}

// Two e4m3 codes as fp16 (h) times 2^e to a bf16 pair: fp16's fields moved to bf16's stand for
// the value times 2^-112 (every code but 0 and NaN is a normal fp16 number), and one bf16
// product with `up` = 2^(112 + e) is exact. For e <= 15 and codes that are not NaN.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h, uint32_t up) {
  const uint32_t b = ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(b), "r"(up));
  return r;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const CopyArgs a) {
  constexpr int kPer = D / 8;
  constexpr uint32_t kRow = kE4m3 ? D : 2 * D, kPiece = kRow / kPer;
  const PagedProblem& p = a.p;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) report_bad_spans(p);
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long at = unit / a.slices;
  if (at >= p.T) return;
  const int t = (int)at;
  int c0 = (int)(unit % a.slices) * a.per_warp * kChunksPerWarp;
  const int c_end = imin(c0 + a.per_warp * kChunksPerWarp, 2 * p.Hkv * kPer);
  int b, pos;
  if (!locate(p, t, lane, b, pos)) return;
  const long long row0 = cache_row(p, b, pos, 0);
  if (row0 < 0) {
    if (lane == 0) atomicOr(p.status, DEV_BAD_INPUT);
    return;
  }
  const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache) + row0 * kRow + lane % kPer * kPiece;
  const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache) + row0 * kRow + lane % kPer * kPiece;
  const uint8_t* ec = kE4m3 ? p.kv_exp + row0 * 2 : nullptr;
  const size_t out_row = (size_t)t * p.Hkv * kPer + lane % kPer;
  uint4* ko = reinterpret_cast<uint4*>(a.out[0]) + out_row;
  uint4* vo = reinterpret_cast<uint4*>(a.out[1]) + out_row;
  for (; c0 < c_end; c0 += kChunksPerWarp) {
    const Pieces<D> pieces(c0, lane, p.Hkv);
    uint4 w[kPieces];
    uint32_t byte[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      int head;
      bool is_v;
      w[j] = make_uint4(0, 0, 0, 0);
      byte[j] = 0;
      if (!pieces.get(j, head, is_v)) continue;
      const uint32_t down = (uint32_t)(head * p.page_size);
      const uint8_t* src = (is_v ? vc : kc) + (size_t)down * kRow;
      if constexpr (kE4m3) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
        w[j].x = x.x;
        w[j].y = x.y;
        byte[j] = __ldg(ec + down * 2ull + is_v);
      } else {
        w[j] = __ldg(reinterpret_cast<const uint4*>(src));
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      int head;
      bool is_v;
      const bool ok = pieces.get(j, head, is_v);
      if constexpr (kE4m3) {
        uint32_t h[4];
        decode4(w[j].x, h[0], h[1]);
        decode4(w[j].y, h[2], h[3]);
        // a byte 0x7F or 0xFF of the codes carries into its top bit
        const uint32_t k = 0x7F7F7F7Fu, one = 0x01010101u;
        const bool nan = (((w[j].x & k) + one) | ((w[j].y & k) + one)) & 0x80808080u;
        if (__any_sync(0xffffffffu, nan || byte[j] > 142u)) {  // NaN, or e > 15: through fp32
          const float s = exp_byte_scale(byte[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = f16x2_to_float2(h[i]);
            h[i] = pack_bf16x2(f.x * s, f.y * s);
          }
        } else {
          const uint32_t up = (byte[j] + 112u) * 0x00800080u;  // 2^(112 + e), twice
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = f16x2_to_bf16x2(h[i], up);
        }
        w[j] = make_uint4(h[0], h[1], h[2], h[3]);
      }
      if (ok) (is_v ? vo : ko)[head * kPer] = w[j];
    }
  }
}

cudaError_t launch_copy(const CopyArgs& args, bool write, cudaStream_t st) {
  const PagedProblem& p = args.p;
  CopyArgs a = args;
  const int chunks = 2 * p.Hkv * (p.d / 8);
  if (p.T == 0 || chunks == 0) return cudaSuccess;
  // A few rows (a decode step) are spread over as many warps as there are slices; long
  // batches give a warp a whole row, whose sequence and slot it looks up once: both kernels
  // are bound by their instructions then (prompts of 29000 tokens: 41 us a slice per warp, 38 us now).
  const int all = ceil_div(chunks, kChunksPerWarp);
  a.per_warp = (long long)p.T * all > 16384 ? all : 1;
  a.slices = ceil_div(all, a.per_warp);
  const long long blocks = ((long long)p.T * a.slices + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)blocks, t = kWarps * 32;
  const bool e = p.e4m3;
  if (write) {
    if (p.d == 64) e ? cache_write_kernel<64, true><<<g, t, 0, st>>>(a) : cache_write_kernel<64, false><<<g, t, 0, st>>>(a);
    else e ? cache_write_kernel<128, true><<<g, t, 0, st>>>(a) : cache_write_kernel<128, false><<<g, t, 0, st>>>(a);
  } else {
    if (p.d == 64) e ? cache_read_kernel<64, true><<<g, t, 0, st>>>(a) : cache_read_kernel<64, false><<<g, t, 0, st>>>(a);
    else e ? cache_read_kernel<128, true><<<g, t, 0, st>>>(a) : cache_read_kernel<128, false><<<g, t, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const PagedProblem& p, const RowView& k, const RowView& v,
                               cudaStream_t st) {
  CopyArgs a{};
  a.p = p;
  a.in[0] = k;
  a.in[1] = v;
  return launch_copy(a, true, st);
}

cudaError_t launch_cache_read(const PagedProblem& p, __nv_bfloat16* k, __nv_bfloat16* v,
                              cudaStream_t st) {
  CopyArgs a{};
  a.p = p;
  a.out[0] = k;
  a.out[1] = v;
  return launch_copy(a, false, st);
}

}  // namespace attn
