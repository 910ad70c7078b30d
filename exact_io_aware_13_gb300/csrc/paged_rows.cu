// Few query rows per kv head over an e4m3 paged cache (decode, speculative tokens, chunks
// of a handful of tokens): each warp streams key tiles of its own.
//
// The recurrence is the forward's ("FlashAttention/es", "El algoritmo FlashAttention"). The
// work is reading 2 (d + 1) bytes per key and kv head once, with 4 d FLOPs per row on top,
// so the kernel is built around the stream:
//   * a CTA (4 warps) takes one key chunk of one (sequence, kv head); warp w takes its
//     32-key tiles w, w + 4, ... through a ring of its own, filled by TMA (codes, one box
//     per page piece) and bulk copies (exponents), and waits for nobody. With 17 to 32 rows
//     two warps share each tile and take 16 rows each (one warp's O would not fit its
//     registers);
//   * codes become fp16 in registers (exact, one conversion for two values) and feed
//     mma.sync m16n8k16 with the KEYS (S^T = K Q^T) or the head dimension (O^T = V^T P^T) as
//     the 16-row side and 8 query rows as the other: with a few query rows per kv head a
//     128-row tile would be empty for the most part. The tensor pipe is not what bounds
//     this: 8 rows at the full HBM rate need about a tenth of the warp-level MMA rate;
//   * MMA slots are permuted so that a thread's fragment bytes are contiguous 16-byte pieces:
//     the head dimension of S^T = K Q^T (K and Q alike), the keys (the order of P^T's columns
//     is the order of V^T's), and the head dimension of O^T (undone when O is written).
//     With the 128-byte swizzle every such shared-memory read is free of bank conflicts;
//   * P^T's fragment is S^T's, transposed by movmatrix: no shared memory in between.
//
// Measured: decode of 64 sequences of 512 to 8192 tokens (Hq = 32, Hkv = 8, d = 128) 94 us with
// the merge, 5.5 TB/s of HBM (81 % of the copy rate); the kernel alone under ncu 92 us. Two
// sequences of 131072: 100 us. 8 new tokens of 16 sequences (32 rows): 225 us, of which 216 in
// the kernel. That is the latency of a warp's steps, with the eight warps per SM that 240
// registers allow: some 2500 clocks per key tile, of which reading, converting and multiplying
// take 1600 and its share of the requests 400, the rest waits. Leaving out every conversion or
// every exponential changed nothing; a quarter of the MMAs with their conversions took 12 %
// off. A CTA's start and end add 8000 clocks to 69000.
//
// Number ranges (fp16 operands, fp32 sums). Q: each row times a power of two that brings its
// largest magnitude to [2^14, 2^15) - exact but for elements below 2^-29 of it, which lose
// bits below 2^-39 of it. P: 2^(s - m + 11) <= 2^15 (the running maximum m may lag by 2^4),
// so weights keep fp16's 11 bits down to 2^-25 of the largest. The V scales are powers of
// two: key j counts 2^(e_j - E) <= 1, E the largest V exponent so far, and O carries 2^E; the
// row sum keeps the plain weights. While all of a tile's scales lie within 2^8 of 2^E, P takes
// that factor and keeps its bits down to 2^-17 of the largest weight at least. In the other
// tiles (one V row of a large norm is enough) V's codes take up to 2^-15 of it, exactly, and P
// what is beyond: with all of it on P, the tail of a long sequence beside one large V row lost
// its weights.
#include <type_traits>

#include "paged.cuh"
#include "paged_out.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 32;        // keys per ring stage
constexpr float kPOffset = 11.0f;  // P is scaled by 2^11
constexpr float kLag = 4.0f;       // O is rescaled when the maximum grows by more than 2^4
constexpr int kNear = 8;           // V scales down to 2^-8 of the largest go to P alone
constexpr int kVDown = 15;         // beyond, V's codes take up to 2^-15 (exact in fp16)

// Key tiles of a CTA in its rings, 8.1 KB each at d = 128: three CTAs fit an SM.
constexpr int kRingTiles = 8;

template <int D>
struct Layout {
  static constexpr int kCodes = kTile * D;                    // one K or V tile
  static constexpr int kStage = 2 * kCodes;                   // swizzled: 1024-byte aligned
  static constexpr int kRing = kRingTiles * kStage;
  static constexpr int kExp = kRing;                          // exponents [tile][32][2]
  static constexpr int kBars = kExp + kRingTiles * kTile * 2;
  static constexpr int kAlloc = kBars + kRingTiles * 8 + 16 + 1024;
};

// Fragment row g (0..7) of a key tile holds key kappa(g): rows g and g + 1 differ in bit 2
// of the key, so the eight lanes of a 16-byte shared-memory phase hit eight swizzled pieces.
__device__ __forceinline__ int kappa(int g) { return (g >> 1) | ((g & 1) << 2); }

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// Offset of 16-byte piece `piece` of row `row` in a swizzled tile of D-byte rows. Rows 8
// apart have the same swizzle.
template <int D>
__device__ __forceinline__ uint32_t piece_offset(int row, int piece) {
  return D == 128 ? row * 128 + ((piece ^ (row & 7)) << 4)
                  : row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
// NT: 8-row groups per warp; RG: warps that share a key tile, each with NT * 8 rows. Three CTAs
// per SM where 168 registers hold a warp's state: d = 64 at NT = 2 216 -> 190 us (32 rows) and
// 118 -> 97 us (16 rows) against two; d = 128 at NT = 2 would spill.
template <int D, int NT, int RG>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 || D == 64 ? 3 : 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedAttention a) {
  using L = Layout<D>;
  constexpr int kSteps = D / 16;   // MMA steps over the head dimension; also 16-row O tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const PagedProblem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  constexpr int kKeyGroups = kWarps / RG, kStages = kRingTiles / kKeyGroups;
  constexpr int kTurns = 6;  // release barriers of a pair
  static_assert(RG == 1 || (RG == 2 && kStages % 2 == 0 && kKeyGroups * kTurns < 16), "named barriers");
  const int kg = warp / RG, rg = warp % RG, row0 = rg * NT * 8;  // key group, first row
  if (blockIdx.x == 0) report_bad_spans(p);
  const int cc = (int)(blockIdx.x % a.n_chunks);
  const int bh = (int)(blockIdx.x / a.n_chunks);
  const int b = bh / p.Hkv, hk = bh - b * p.Hkv;
  const Span sp = load_span(p, b);
  const int rows = sp.n * a.G;  // packed row i * G + g of query token i, head hk * G + g
  if (rows == 0) return;
  // Keys of the chunk that any row sees: the first token's lower end, the last one's upper.
  int lo0, hi0, lo1, hi1;
  decode_row_keys(a.mask_kind, a.window, sp.L, sp.n, 0, lo0, hi0);
  decode_row_keys(a.mask_kind, a.window, sp.L, sp.n, sp.n - 1, lo1, hi1);
  const int k_lo = imax(lo0, cc * a.chunk);
  const int k_hi = imin(hi1, (int)imin64((long long)(cc + 1) * a.chunk, sp.L));
  if (k_hi <= k_lo && a.n_chunks > 1) return;  // the merge reads no such chunk
  const int tb = k_lo / kTile, te = k_hi > k_lo ? ceil_div(k_hi, kTile) : tb;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int* abort_flag = reinterpret_cast<int*>(smem + L::kBars + kRingTiles * 8);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRingTiles; ++i) mbar_init(smem_u32(bars + i), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const WaitCtx wc{abort_flag, p.status};
  const uint32_t ring = smem_u32(smem) + kg * kStages * L::kStage;
  const uint32_t exps = smem_u32(smem + L::kExp) + kg * kStages * kTile * 2;
  const uint32_t full = smem_u32(bars) + kg * kStages * 8;

  // The query rows' loads are on their way while the first tiles are requested.
  uint32_t qw[NT][kSteps][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = row0 + nt * 8 + g;
    const bool ok = r < rows;
    const int i = ok ? r / a.G : 0, h = hk * a.G + (ok ? r - i * a.G : 0);
    const long long t = p.offsets ? sp.row0 + i : i;
    const __nv_bfloat16* q = a.q + (p.offsets ? 0 : b) * a.q_batch + t * a.q_token + h * a.q_head;
#pragma unroll
    for (int v = 0; v < kSteps / 2; ++v) {  // 16-byte loads: two steps each
      uint4 x = make_uint4(0, 0, 0, 0);
      if (ok) x = __ldg(reinterpret_cast<const uint4*>(q + (v >> 1) * 64 + c * 16 + (v & 1) * 8));
      qw[nt][2 * v][0] = x.x; qw[nt][2 * v][1] = x.y;
      qw[nt][2 * v + 1][0] = x.z; qw[nt][2 * v + 1][1] = x.w;
    }
  }

  // Requests this warp's next tile into stage s: lane q fetches its q-th page piece, whose
  // page-table entry it loaded at the request before. The warps of a pair take turns (kStages
  // is even, so a stage stays with its warp): a request costs 600 clocks, a tile 1600.
  const int R = imin(p.page_size, kTile), pieces = kTile / R;
  constexpr int kStride = kKeyGroups * RG * kTile;
  int key = (tb + kg + kKeyGroups * rg) * kTile + lane * R;
  PageWalk walk(key, p.page_size);
  const int32_t* table = p.page_table + (size_t)b * p.max_pages;
  auto wanted = [&] { return lane < pieces && key < sp.L && key + R > k_lo; };
  int page = wanted() ? __ldg(table + walk.page) : -1;
  auto request = [&](int s) {
    int row = -1;
    if (wanted()) {
      row = (int)paged_row(page, p.num_pages, p.Hkv, p.page_size, hk, walk.slot);
      if (row < 0) atomicOr(p.status, DEV_BAD_INPUT);
    }
    const uint32_t bar = full + s * 8;
    const uint32_t n = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0));
    if (lane == 0) mbar_arrive_expect_tx(bar, n * R * (2 * D + 2));
    __syncwarp();
    if (row >= 0) {
      const uint32_t kt = ring + s * L::kStage + lane * R * D;
      tma_load_2d(kt, &tm_k, bar, 0, row);
      tma_load_2d(kt + L::kCodes, &tm_v, bar, 0, row);
      bulk_load(exps + (s * kTile + lane * R) * 2, p.kv_exp + (size_t)row * 2, R * 2, bar);
    }
    key += kStride;
    walk.advance(kStride, p.page_size);
    page = wanted() ? __ldg(table + walk.page) : -1;
  };
  int issued = tb + kg + kKeyGroups * rg;  // next tile to request
  for (int s = rg; s < kStages && issued < te; s += RG, issued += kKeyGroups * RG) request(s);

  // Q fragments: thread (g, c) holds, of row nt * 8 + g, the head dimensions 16 c + 4 s .. + 3
  // (and 64 + ... for steps 4-7) of step s, the pieces it reads of K.
  uint32_t qf[NT][kSteps][2];
  float k1[NT][2], slope[NT][2];
  int lo[NT][2], hi[NT][2], pos[NT][2];
  const float unit = (a.score_kind & ATTN_SCORE_SOFTCAP) ? 1.0f / a.softcap : kPagedLog2e;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t (&w)[kSteps][2] = qw[nt];
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) top = max(top, max(w[s][e] & 0x7FFFu, (w[s][e] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // top = m 2^x, 1 <= m < 2; the row times 2^(14 - x). Rows below 2^-112 keep x = -112.
    const int x = imax((int)(top >> 7) - 127, -112);
    const float up = __uint_as_float((uint32_t)(14 - x + 127) << 23);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qf[nt][s][e] = pack_f16x2(__uint_as_float(w[s][e] << 16) * up,
                                  __uint_as_float(w[s][e] & 0xFFFF0000u) * up);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // the softmax's rows of this thread: nt * 8 + 2 c + e
      const int rr = row0 + nt * 8 + 2 * c + e;
      const int xr = __shfl_sync(0xffffffffu, x, (2 * c + e) * 4);
      const int ii = rr / a.G, hh = hk * a.G + rr - ii * a.G;
      // 2^(xr - 14) is a normal number: xr >= -112
      k1[nt][e] = a.scale * unit * __uint_as_float((uint32_t)(xr - 14 + 127) << 23);
      slope[nt][e] = (a.score_kind & ATTN_SCORE_ALIBI) ? alibi_slope(hh, a.Hq) * unit : 0.f;
      lo[nt][e] = hi[nt][e] = 0;
      if (rr < rows) decode_row_keys(a.mask_kind, a.window, sp.L, sp.n, ii, lo[nt][e], hi[nt][e]);
      pos[nt][e] = sp.L - sp.n + ii;
    }
  }

  float o[NT][kSteps][4];  // O^T: (dims of fragment rows g, g + 8) x (query rows 2 c, 2 c + 1)
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][s][e] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }
  int E = 0;  // largest V exponent byte so far
  const bool plain = !(a.score_kind & (ATTN_SCORE_ALIBI | ATTN_SCORE_SOFTCAP));
  const float cap = a.softcap * kPagedLog2e;

  // This lane's offsets in the tiles: K pieces c and 4 + c of key row kappa(g), V pieces of
  // key rows c and c + 4.
  uint32_t koff[D / 64], voff[2];
#pragma unroll
  for (int half = 0; half < D / 64; ++half) koff[half] = piece_offset<D>(kappa(g), half * 4 + c);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    voff[k] = L::kCodes + (D == 128 ? piece_offset<D>(c + 4 * k, kappa(g))
                                    : piece_offset<D>(c + 4 * k, g >> 1) + (g & 1) * 8);

  bool live = true;
  int s = 0;
  uint32_t parity = 0;
  // A pair releases its i-th tile through named barrier i % kTurns: the warp that will not
  // refill the stage arrives when it has read the tile, the one that will waits there after
  // its next tile, so that neither waits for the other's request. Neither gets more than two
  // tiles ahead (an arrival is followed by a wait for the other's), so at most five
  // consecutive barriers are in use. Returns whether this warp refills the stage before.
  int i_tile = 0, turn = 0;
  auto release = [&]() -> bool {
    const int before = turn == 0 ? kTurns - 1 : turn - 1, at = turn;
    turn = turn == kTurns - 1 ? 0 : turn + 1;
    const bool mine = i_tile % RG == rg, first = i_tile == 0;
    ++i_tile;
    if (mine) return false;
    nb_arrive(1 + kg * kTurns + at, RG * 32);
    if (first) return false;
    nb_sync(1 + kg * kTurns + before, RG * 32);
    return true;
  };
  for (int tile = tb + kg; tile < te; tile += kKeyGroups) {
    if (live) live = __all_sync(0xffffffffu, mbar_wait(full + s * 8, parity, wc));
    if (!live) {  // keep the barriers of the warps that share the tile paired
      if (RG > 1) release();
      continue;
    }
    const int t0 = tile * kTile;
    const uint32_t kt = ring + s * L::kStage, vt = kt + L::kCodes, et = exps + s * kTile * 2;
    const int valid = imin(kTile, sp.L - t0);
    // Slots behind the sequence and keys that were not loaded: their V must not reach the sums.
    const int skip = paged_skipped_keys(t0, k_lo, R);
    if (valid < kTile || skip > 0) {
      for (int e = lane; e < kTile * (D / 16); e += 32) {
        const int row = e / (D / 16), piece = e % (D / 16);
        const uint32_t at = vt + piece_offset<D>(row, piece);
        if (row < skip || row >= valid)
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
      }
      fence_proxy_async_smem();  // the first tile's stage is refilled by TMA
      __syncwarp();  // (warps that share the tile write the same zeros before they read it)
    }
    const uint32_t e_lane = lds16(et + lane * 2) >> 8;  // V exponent of key t0 + lane
    const bool seen = t0 + lane >= k_lo && t0 + lane < k_hi;  // by some row
    const int Et = (int)__reduce_max_sync(0xffffffffu, seen ? e_lane : 0u);
    const int E_min = (int)__reduce_min_sync(0xffffffffu, seen && e_lane ? e_lane : 255u);
    // Whether every row sees every key of the tile (warp-uniform)
    const bool masked = t0 < lo1 || t0 + kTile > hi0;

    // ---- S^T = K Q^T for the two 16-key halves
    // The MMAs of a chain depend on one another (35 clocks each): both key halves, and for
    // one row group both halves of the head dimension, run as chains of their own.
    constexpr int kSplit = NT == 1 ? D / 64 : 1;
    float xs[kSplit][2][NT][4];
#pragma unroll
    for (int q = 0; q < kSplit; ++q)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) xs[q][hf][nt][e] = 0.f;
#pragma unroll
    for (int h0 = 0; h0 < D / 64; h0 += kSplit) {
      uint4 ku[kSplit][2], kv[kSplit][2];
#pragma unroll
      for (int q = 0; q < kSplit; ++q)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          ku[q][hf] = lds128(kt + koff[h0 + q] + hf * 16 * D);
          kv[q][hf] = lds128(kt + koff[h0 + q] + (hf * 16 + 8) * D);
        }
#pragma unroll
      for (int st = 0; st < 4; ++st)
#pragma unroll
        for (int q = 0; q < kSplit; ++q)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t uw[4] = {ku[q][hf].x, ku[q][hf].y, ku[q][hf].z, ku[q][hf].w};
            const uint32_t vw[4] = {kv[q][hf].x, kv[q][hf].y, kv[q][hf].z, kv[q][hf].w};
            uint32_t a0, a1, a2, a3;
            decode4(uw[st], a0, a2);
            decode4(vw[st], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(xs[q][hf][nt], a0, a1, a2, a3, qf[nt][(h0 + q) * 4 + st][0], qf[nt][(h0 + q) * 4 + st][1]);
          }
    }
    float x[2][NT][4], ks[2][2];
    int ve[2][2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[hf][nt][e] = kSplit == 2 ? xs[0][hf][nt][e] + xs[kSplit - 1][hf][nt][e] : xs[0][hf][nt][e];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w = lds16(et + (hf * 16 + kappa(g) + 8 * e) * 2);
        ks[hf][e] = exp_byte_scale(w & 255u);
        ve[hf][e] = (int)(w >> 8);
      }
    }
    // ---- scores in log2 units (rows 2 c, 2 c + 1 of a key in one packed pair), row maxima.
    // Every decision is warp-uniform and stays outside the element loops.
    float mt[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mt[nt][0] = mt[nt][1] = -INFINITY;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          f32x2_split(mul_f32x2(f32x2(x[hf][nt][2 * e], x[hf][nt][2 * e + 1]),
                                mul_f32x2(f32x2(k1[nt][0], k1[nt][1]), f32x2(ks[hf][e], ks[hf][e]))),
                      x[hf][nt][2 * e], x[hf][nt][2 * e + 1]);
    if (!plain) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = t0 + hf * 16 + kappa(g) + 8 * e;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) x[hf][nt][2 * e + r] -= slope[nt][r] * (float)(pos[nt][r] - j);
        }
      if (a.score_kind & ATTN_SCORE_SOFTCAP) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[hf][nt][e] = cap * tanhf(x[hf][nt][e]);
      }
    }
    if (masked) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = t0 + hf * 16 + kappa(g) + 8 * e;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (j < lo[nt][r] || j >= hi[nt][r]) x[hf][nt][2 * e + r] = -INFINITY;
        }
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) mt[nt][e & 1] = fmaxf(mt[nt][e & 1], x[hf][nt][e]);
    bool grow = Et > E;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          mt[nt][r] = fmaxf(mt[nt][r], __shfl_xor_sync(0xffffffffu, mt[nt][r], off));
        grow |= mt[nt][r] > m[nt][r] + kLag;
      }
    if (__any_sync(0xffffffffu, grow)) {
      const int En = imax(E, Et);
      const float fe = En - E > 126 ? 0.f : __uint_as_float((uint32_t)(127 - (En - E)) << 23);
      E = En;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float mn = fmaxf(m[nt][r], mt[nt][r]);
          const float f = mn == -INFINITY ? 1.f : ex2_approx(m[nt][r] - mn);
          m[nt][r] = mn;
          l[nt][r] *= f;
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            o[nt][st][r] *= f * fe;
            o[nt][st][2 + r] *= f * fe;
          }
        }
    }
    // Whether P alone cannot take the tile's V scales. (Byte 0, a row of zeros for the most
    // part, is not among E_min; such a row adds nothing beside E > kVDown + kNear.)
    const bool far = E - E_min > kNear || (E > kNear && E <= kVDown + kNear);
    // ---- P^T (fp16) and O^T += V^T P^T
    uint64_t off2[NT], l2[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      off2[nt] = f32x2(m[nt][0] == -INFINITY ? 0.f : kPOffset - m[nt][0],
                       m[nt][1] == -INFINITY ? 0.f : kPOffset - m[nt][1]);
      l2[nt] = f32x2(l[nt][0], l[nt][1]);
    }
    const uint64_t one2 = f32x2(1.f, 1.f);
    // kFar: V's codes take a part of the scales. (One branch around both key halves: inside, it
    // keeps the second half's exponentials from running beside the first half's MMAs, and 8 new
    // tokens of 16 sequences take 236 us instead of 233.)
    auto add_pv = [&](auto is_far) {
      constexpr bool kFar = decltype(is_far)::value;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pf[NT][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // V scale relative to 2^E (0 for the smallest; at most 1, also for keys that no row
          // sees, whose bytes are anything and whose P is 0)
          const int down = E - ve[hf][e] - (kFar ? kVDown : 0);
          const float wj = __uint_as_float((uint32_t)imax(127 - imax(down, 0), 0) << 23);
          const uint64_t wj2 = f32x2(wj, wj);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p0, p1;
            f32x2_split(fma_f32x2(f32x2(x[hf][nt][2 * e], x[hf][nt][2 * e + 1]), one2, off2[nt]), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            l2[nt] = fma_f32x2(f32x2(p0, p1), one2, l2[nt]);
            f32x2_split(mul_f32x2(f32x2(p0, p1), wj2), p0, p1);
            pf[nt][e] = transpose_8x8(pack_f16x2(p0, p1));
          }
        }
        // keys of the transposed fragment's slots 2 c, 2 c + 1: c, c + 4 (and + 8)
        uint32_t w[4][D / 32], f01 = 0, f23 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t at = kt + voff[k & 1] + (hf * 16 + 8 * (k >> 1)) * D;
          if constexpr (D == 128) {
            const uint4 v = lds128(at);
            w[k][0] = v.x; w[k][1] = v.y; w[k][2] = v.z; w[k][3] = v.w;
          } else {
            const uint2 v = lds64(at);
            w[k][0] = v.x; w[k][1] = v.y;
          }
        }
        if constexpr (kFar) {
          auto factor = [&](int k) {  // V's part of the scale of key hf * 16 + k
            const int down = E - (int)(lds16(et + (hf * 16 + k) * 2) >> 8);
            return __uint_as_float((uint32_t)(127 - imin(imax(down, 0), kVDown)) << 23);
          };
          f01 = pack_f16x2(factor(c), factor(c + 4));
          f23 = pack_f16x2(factor(c + 8), factor(c + 12));
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {  // two head dimensions of the word: one O tile
            const uint32_t sel = hb ? 0x7362u : 0x5140u;
            const uint32_t u = prmt(w[0][i], w[1][i], sel), v = prmt(w[2][i], w[3][i], sel);
            uint32_t a0, a1, a2, a3;
            decode4(u, a0, a1);
            decode4(v, a2, a3);
            if constexpr (kFar) {
              a0 = mul_f16x2(a0, f01); a1 = mul_f16x2(a1, f01);
              a2 = mul_f16x2(a2, f23); a3 = mul_f16x2(a3, f23);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(o[nt][2 * i + hb], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
          }
      }
    };
    if (far) add_pv(std::true_type{});
    else add_pv(std::false_type{});
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) f32x2_split(l2[nt], l[nt][0], l[nt][1]);
    __syncwarp();  // every thread has read the stage
    if ((RG == 1 || release()) && issued < te) {
      request(RG == 1 ? s : s == 0 ? kStages - 1 : s - 1);
      issued += kKeyGroups * RG;
    }
    if (++s == kStages) {
      s = 0;
      parity ^= 1;
    }
  }
  if (RG > 1 && i_tile > 0 && (i_tile - 1) % RG == rg)  // the other's last arrival
    nb_sync(1 + kg * kTurns + (turn == 0 ? kTurns - 1 : turn - 1), RG * 32);
  if (!live)  // leave no copy in flight into this CTA's shared memory
    for (int i = 0; i < kStages; ++i) drain_wait(full + i * 8, i < s ? parity ^ 1 : parity);

  // ---- merge of the key groups: factors 2^(m_k - M) 2^E_k, fixed order. 2^E_k comes after the
  // division by the row sum: V may lie near the top of fp32's range, and O carries 2^11 and the
  // sum until then.
  grid_dependents_launch();
  __syncthreads();
  constexpr int kRows = NT * 8 * RG;
  float* sm_m = reinterpret_cast<float*>(smem);            // [key group][row]
  float* sm_l = sm_m + kKeyGroups * kRows;
  float* sm_o = sm_l + kKeyGroups * kRows;                 // [key group][row][D + 4]
  float* sm_v = sm_o + kKeyGroups * kRows * (D + 4);       // [warp]: 2^E_k
  static_assert(((2 + D + 4) * kKeyGroups * kRows + kWarps) * 4 <= L::kRing, "merge space");
  if (lane == 0) sm_v[warp] = exp_byte_scale((uint32_t)E);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float sum = l[nt][r];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const int rr = kg * kRows + row0 + nt * 8 + 2 * c + r;
      if (g == 0) {
        sm_m[rr] = m[nt][r];
        sm_l[rr] = sum;
      }
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int dim = D == 128 ? 16 * kappa(g) + 2 * st : 8 * g + 2 * st;
        *reinterpret_cast<float2*>(sm_o + rr * (D + 4) + dim) =
            make_float2(o[nt][st][r], o[nt][st][2 + r]);
      }
    }
  __syncthreads();
  const bool ok = *abort_flag == 0;
  // Warp w finishes rows w, w + 4, ...: lane k does the scalar work of the k-th (one row after
  // the other it took 830 clocks each, 7 % of a CTA with 32 rows), then all lanes sum them up.
  constexpr int kMine = kRows / kWarps;
  float fk[kKeyGroups], l2 = -INFINITY;
  int i_row = 0, h_row = 0;
  {
    const int rr = warp + kWarps * imin(lane, kMine - 1);
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kKeyGroups; ++k) M = fmaxf(M, sm_m[k * kRows + rr]);
#pragma unroll
    for (int k = 0; k < kKeyGroups; ++k) {
      const float mk = sm_m[k * kRows + rr];
      fk[k] = mk == -INFINITY || !ok ? 0.f : ex2_approx(mk - M);
      sum = fmaf(fk[k], sm_l[k * kRows + rr], sum);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (a NaN sum makes the row NaN)
#pragma unroll
    for (int k = 0; k < kKeyGroups; ++k) fk[k] *= inv;
    if (sum != 0.f) l2 = M - kPOffset + log2f(sum);
    i_row = rr / a.G;
    h_row = hk * a.G + rr - i_row * a.G;
  }
#pragma unroll 2
  for (int n = 0; n < kMine; ++n) {
    const int rr = warp + kWarps * n;
    if (rr >= rows) break;
    float acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < kKeyGroups; ++k) {
      const float f = __shfl_sync(0xffffffffu, fk[k], n);
      const float vs = sm_v[k * RG];  // (the warps of a pair have seen the same scales)
      const float* src = sm_o + (k * kRows + rr) * (D + 4) + lane * (D / 32);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] = f != 0.f ? fmaf(f * src[e], vs, acc[e]) : acc[e];
    }
    const int i = __shfl_sync(0xffffffffu, i_row, n), h = __shfl_sync(0xffffffffu, h_row, n);
    store_row<D>(a, b, sp.row0 + i, i, h, cc, lane, acc, __shfl_sync(0xffffffffu, l2, n));
  }
}

template <int D, int NT, int RG>
cudaError_t launch_nt(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st) {
  auto kern = paged_rows_kernel<D, NT, RG>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Layout<D>::kAlloc, done);
  if (e != cudaSuccess) return e;
  const long long grid = (long long)a.p.B * a.p.Hkv * a.n_chunks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, kWarps * 32, Layout<D>::kAlloc, st>>>(maps.k, maps.v, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st) {
  const int rows = a.p.max_new * a.G;
  if (rows <= 8) return launch_nt<D, 1, 1>(a, maps, st);
  if (rows <= 16) return launch_nt<D, 2, 1>(a, maps, st);
  return launch_nt<D, 2, 2>(a, maps, st);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st) {
  return a.p.d == 64 ? launch_d<64>(a, maps, st) : launch_d<128>(a, maps, st);
}

}  // namespace attn
