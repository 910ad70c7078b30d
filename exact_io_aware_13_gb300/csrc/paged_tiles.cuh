// Attention of packed rows over the paged cache on the fifth-generation tensor cores:
// chunks of new tokens (prefill), and decode with more rows per kv head than
// paged_rows.cu takes.
//
// The algorithm is the forward kernel's (fwd_tc.cu: tiled online softmax, two 128-row query
// tiles against 128-key tiles, S and O in tensor memory, P written over S). What differs:
//   * rows are packed: row r of a (sequence, kv head) is query token r / G, query head
//     hk * G + r % G, so every key tile serves the whole group and a short chunk still fills
//     the 128 rows of an MMA. A CTA takes 256 consecutive packed rows of one (sequence, kv
//     head) against one key chunk; the softmax warps bring their Q rows into swizzled shared
//     memory themselves (any strides, any G);
//   * key tiles come from pages: two loader warps (K, V) issue one TMA box (bf16) or bulk
//     copy (codes) per page piece, their page-table entries fetched one tile ahead. Pages of
//     64, 16 and 8 take the long chunk below 1392, 1396 and 1661 us; one warp for both took
//     pages of 16 1.4 times as long as pages of 64;
//   * masks are aligned at the bottom right (decode_row_keys), slots behind the sequence are
//     masked in S and cleared in V, and so are the pages of the first key tile that no row of
//     the unit sees: they are not loaded (a sliding window may have given them back);
//   * a unit of at most 128 rows leaves no second query tile to overlap with, so its even
//     key tiles go to the first softmax warpgroup and its odd ones to the second (two score
//     buffers, two O accumulators), merged at the end;
//   * the key axis may be cut into chunks: fp32 partial rows, merged by their log-sum-exp.
//
// e4m3 cache: a fourth warpgroup converts code tiles to fp16 operand tiles. The scales are
// powers of two, so a K tile becomes code * 2^(e_j - E), E the tile's largest exponent:
// exact down to 2^15 between scales, and off by at most 2^-25 of the largest scale below;
// 2^E multiplies the tile's scores with the softmax scale. A V tile is scaled the same way
// with E_V, and P by 2^(E_V - E_ref), E_ref the largest E_V so far, which O carries (row sums
// keep the plain weights). E_V is taken no smaller than E_ref - 8, so that P keeps its
// range. P = 2^(s - m + 11) in fp16 (11 bits down to 2^-25 of the largest weight, where a
// bf16 P keeps 8), m lagging by at most 2^4; Q rows are scaled by a power of two into
// [2^14, 2^15).
//
// What bounds it, measured (one chunk of 4096 tokens after 28672 cached ones, Hq = 32, Hkv =
// 8, d = 128, 2.06 TFLOP): bf16 1370 to 1416 us in runs that heat the GPU up to its power cap
// (1500 to 1455 TFLOP/s; 1314 us once, with cool clocks), a step of two query tiles against a
// key tile in 2700 clocks where the MMAs alone need 2048: the chain S -> softmax -> P V of a
// tile, as in the forward kernel. e4m3 1827 us = 1128 TFLOP/s: the softmax of a tile takes
// 2160 clocks instead of 1310 beside the converters, whose fp16 tiles also cost 512 clocks of
// shared-memory writes per step (without the conversion: 1440 TFLOP/s). Few rows over long
// caches are bound by HBM (bf16, 32 rows: 5.1 TB/s) or by the conversion (e4m3).
#pragma once

#include "paged.cuh"

namespace attn {
namespace pt {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr int kQTiles = 2;
constexpr int kUnitRows = kQTiles * BM;
constexpr int kLoadKWarp = 8, kMmaWarp = 9, kRelayWarp = 10, kLoadVWarp = 11, kConvWarp = 12;
constexpr int kInfo = 4;             // slots of the converters' per-tile scales
// Named barriers: kNbP + 2 t + part: P_t, or half of it, in tensor memory, softmax warpgroup t
// and the MMA warp; kNbKv + s: operand stage s filled; kNbDual: both softmax warpgroups, before
// a dual unit's merge.
constexpr uint32_t kNbP = 1, kNbPCount = 160;
constexpr uint32_t kNbKv = 5;
constexpr uint32_t kNbDual = 9;
constexpr float kPOffset = 11.0f;    // e4m3: P is scaled by 2^11 (fp16)
constexpr int kMaxDown = 8;          // e4m3: a V tile's exponent is at least E_ref - 8

template <bool kE4m3>
struct Shape {
  static constexpr int kThreads = kE4m3 ? 512 : 384;
  static constexpr int kStages = kE4m3 ? 3 : 4;       // operand tiles in the ring
  // Code tiles on their way or waiting for conversion. A dual unit streams its keys as fast
  // as HBM gives them: it adds the second query tile's room (two code tiles) to its ring.
  static constexpr int kCodeStages = kE4m3 ? 4 : 0, kCodeStagesDual = kE4m3 ? 6 : 0;
  static constexpr uint32_t kNbKvCount = kE4m3 ? 160 : 64;
  // Registers: softmax threads hold 128 scores and the row state, the others little. The
  // launch gives kThreads x kRegsLaunch; the split must not exceed it (launch_variant checks
  // what the compiler used).
  static constexpr int kRegsLaunch = kE4m3 ? 128 : 168;
  static constexpr int kRegsSoftmax = kE4m3 ? 168 : 208;
  static constexpr int kRegsOther = 88;
  static constexpr int kRegsConvert = 88;
  static_assert(256 * kRegsSoftmax + 128 * kRegsOther + (kE4m3 ? 128 * kRegsConvert : 0) <=
                    kThreads * kRegsLaunch,
                "register pool");
  // P is handed to the MMA warp in two halves, so that the first products overlap the second
  // half's exponentials: long chunk 1361 -> 1314 us over bf16 (cool clocks both). Over e4m3, whose softmax warps
  // have fewer registers, six chunks went 689 -> 710 us: one part there.
  static constexpr int kPParts = kE4m3 ? 1 : 2;
  static constexpr float kLag = kE4m3 ? 4.0f : 8.0f;  // O is rescaled beyond this growth (log2)
};

template <int D, bool kE4m3>
struct Layout {
  using S = Shape<kE4m3>;
  static constexpr int kChunk = BM * 128;             // 128 rows of 128 bytes
  static constexpr int kSlabs = D / 64;
  static constexpr int kTile = BM * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + kQTiles * kTile;
  static constexpr int kCodes = kRing + S::kStages * kTile;
  static constexpr int kCodeTile = BN * D;
  static constexpr int kExp = kCodes + S::kCodeStages * kCodeTile;   // [kInfo][128][2]
  static constexpr int kBars = kExp + (kE4m3 ? kInfo * BN * 2 : 0);
  static constexpr int kAlloc = kBars + 512 + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
};
static_assert(Layout<128, true>::kAlloc <= 232448 && Layout<128, false>::kAlloc <= 232448,
              "shared memory");

// Key tiles of one query tile, and the range in which every one of its rows sees every key.
struct TileKeys {
  int lo, hi;            // tiles [lo, hi) of BN keys
  int full_lo, full_hi;  // keys
};

// A CTA's work, found by warp 0 and kept in shared memory: held in every thread's registers
// it would not fit the few that the loader and the converters have.
struct Cta {
  int b, hk, cc;         // sequence (< 0: nothing to do), kv head, key chunk
  int row_base, rows;    // first packed row, packed rows from there on
  int c0, c1;            // keys of the chunk
  int k_lo;              // lowest key that any row sees
  int lo, hi;            // key tiles of both query tiles together
  bool dual;             // one query tile: its key tiles alternate between two streams
  Span span;
  TileKeys tk[kQTiles];
};

struct Bars {
  uint64_t q_full;
  uint64_t kv_full[4];
  uint64_t kv_empty[4];
  uint64_t s_full[kQTiles];
  uint64_t o_full[kQTiles];
  uint64_t code_full[6];
  uint64_t code_empty[6];
  uint64_t info_full[kInfo];
  int4 info[kInfo];     // E_K, E_V, E_ref of key tile j (slot j % kInfo)
  uint32_t tmem_base;
  int abort_flag;
  Cta cta;
};
static_assert(sizeof(Bars) <= 512, "barrier space");

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// CTA -> (sequence, kv head, key chunk, row unit): sequence b owns units_b * Hkv * chunks_b
// consecutive CTAs, the units of one (kv head, chunk) together, so that CTAs running at the
// same time read the same keys from L2; the last units (the longest rows under causal
// masks) come first. One warp, all lanes.
__device__ __forceinline__ void find_work(const PagedAttention& a, Cta* w, int lane) {
  const PagedProblem& p = a.p;
  long long at = blockIdx.x, base = 0;
  if (lane == 0) w->b = -1;
  __syncwarp();
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    Span s{0, 0, 0};
    if (b < p.B) s = load_span(p, b);
    const int units = (int)(((long long)s.n * a.G + kUnitRows - 1) / kUnitRows);
    // (with several chunks the merge writes the rows of an empty sequence)
    const int chunks = a.n_chunks == 1 ? 1 : (int)(((long long)s.L + a.chunk - 1) / a.chunk);
    const long long mine = (long long)units * p.Hkv * chunks;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    const long long first = base + incl - mine;
    const bool hit = at >= first && at < first + mine;
    if (hit) {
      const int rem = (int)(at - first);
      const int u = rem % units, hc = rem / units;
      w->b = b;
      w->hk = hc / chunks;
      w->cc = hc % chunks;
      w->row_base = (units - 1 - u) * kUnitRows;
      w->rows = s.n * a.G - w->row_base;
      w->c0 = a.n_chunks == 1 ? 0 : w->cc * a.chunk;
      w->c1 = a.n_chunks == 1 ? s.L : (int)imin64((long long)w->c0 + a.chunk, s.L);
      w->span = s;
      w->lo = 1 << 30;
      w->k_lo = w->c1;
      w->hi = 0;
      for (int t = 0; t < kQTiles; ++t) {
        TileKeys k{0, 0, 0, 0};
        const int r0 = t * BM;
        if (r0 < w->rows) {
          int la, ha, lb, hb;  // keys of the tile's first and last token
          decode_row_keys(a.mask_kind, a.window, s.L, s.n, (w->row_base + r0) / a.G, la, ha);
          decode_row_keys(a.mask_kind, a.window, s.L, s.n,
                          (w->row_base + imin(r0 + BM, w->rows) - 1) / a.G, lb, hb);
          k.full_lo = imax(lb, w->c0);
          k.full_hi = imin(ha, w->c1);
          const int k_lo = imax(la, w->c0), k_hi = imin(hb, w->c1);
          if (k_hi > k_lo) {
            k.lo = k_lo / BN;
            k.hi = (k_hi + BN - 1) / BN;
            w->lo = imin(w->lo, k.lo);
            w->k_lo = imin(w->k_lo, k_lo);
            w->hi = imax(w->hi, k.hi);
          }
        }
        w->tk[t] = k;
      }
      w->dual = w->rows <= BM && w->hi - w->lo >= 2;
    }
    if (__any_sync(0xffffffffu, hit)) return;
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <int D, bool kAlibi, bool kSoftcap, bool kE4m3>
__global__ void __launch_bounds__(Shape<kE4m3>::kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedAttention a) {
  using S = Shape<kE4m3>;
  using L = Layout<D, kE4m3>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const PagedProblem& p = a.p;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (blockIdx.x == 0) report_bad_spans(p);
  if (warp == 0) find_work(a, &bars->cta, lane);
  if (threadIdx.x == 32) {
    mbar_init(smem_u32(&bars->q_full), 8);  // one arrival per softmax warp
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&bars->kv_full[s]), 1);
      mbar_init(smem_u32(&bars->kv_empty[s]), 1);
    }
    for (int s = 0; s < S::kCodeStagesDual; ++s) {
      mbar_init(smem_u32(&bars->code_full[s]), 1);
      mbar_init(smem_u32(&bars->code_empty[s]), 4);  // one arrival per converter warp
    }
    for (int s = 0; s < kInfo; ++s) mbar_init(smem_u32(&bars->info_full[s]), 1);
    for (int t = 0; t < kQTiles; ++t) {
      mbar_init(smem_u32(&bars->s_full[t]), 1);
      mbar_init(smem_u32(&bars->o_full[t]), 1);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const Cta& w = bars->cta;
  if (w.b < 0) return;

  // Packed row r of this unit: its token (index among the new ones, packed row) and head.
  struct Row {
    int i, t, h;
  };
  auto row_of = [&](int r) {
    const int pr = w.row_base + r, i = pr / a.G;
    return Row{i, w.span.row0 + i, w.hk * a.G + pr - i * a.G};
  };
  auto q_row = [&](const Row& x) {
    return a.q + (p.offsets ? 0 : w.b) * a.q_batch + (p.offsets ? x.t : x.i) * a.q_token + x.h * a.q_head;
  };
  auto o_row = [&](const Row& x) {
    return a.o + (p.offsets ? 0 : w.b) * a.o_batch + (p.offsets ? x.t : x.i) * a.o_token + x.h * a.o_head;
  };
  auto lse_row = [&](const Row& x) {
    return a.lse + (p.offsets ? 0 : w.b) * a.l_batch + (p.offsets ? x.t : x.i) * a.l_token + x.h * a.l_head;
  };

  if (w.hi <= w.lo) {  // no row sees a key of this chunk
    if (a.n_chunks > 1) return;  // the merge reads no such chunk
    for (int r = threadIdx.x; r < imin(kUnitRows, w.rows); r += S::kThreads) {
      const Row x = row_of(r);
      uint4* dst = reinterpret_cast<uint4*>(o_row(x));
#pragma unroll
      for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
      *lse_row(x) = -INFINITY;
    }
    return;
  }

  // Code stage s (e4m3): the ones past kCodeStages lie in the second query tile's room.
  auto code_tile = [&](int s) {
    return smem + (s < S::kCodeStages ? L::kCodes + s * L::kCodeTile
                                      : L::kQ + L::kTile + (s - S::kCodeStages) * L::kCodeTile);
  };

  // Page pieces: keys of one copy. Those of the first key tile that lie wholly below every
  // row's keys are not loaded.
  auto piece_keys = [&] { return kE4m3 && p.page_size % 128 == 0 ? 128 : imin(p.page_size, 64); };
  auto skipped = [&] { return paged_skipped_keys(w.lo * BN, w.k_lo, piece_keys()); };

  WaitCtx wc{&bars->abort_flag, p.status};
  // The softmax warps request their Q rows before the loader starts: behind its stream of
  // keys they would take several times as long.
  constexpr int kPer = D / 8, kRowsPerIter = 32 / kPer, kQIters = 32 / kRowsPerIter;
  const int wt = (warp >> 2) & 1;                                // query tile of a softmax warp
  const int wrow = (w.dual ? 0 : wt * BM) + (warp & 3) * 32;     // its first row in the unit
  uint4 qv[kQIters];
  if (warp < 8) {
#pragma unroll
    for (int it = 0; it < kQIters; ++it) {
      const int rr = wrow + it * kRowsPerIter + lane / kPer;
      qv[it] = make_uint4(0, 0, 0, 0);
      if (rr < w.rows) qv[it] = __ldg(reinterpret_cast<const uint4*>(q_row(row_of(rr))) + lane % kPer);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&bars->tmem_base), L::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;

  if (kE4m3 && warp >= kConvWarp) {
    setmaxnreg_dec<S::kRegsConvert>();
    // ------------------------------------------------------------ converters (e4m3)
    // A warp converts 32 of a tile's rows, 256 codes at a time: a lane turns eight codes (one
    // 8-byte read) into one 16-byte column of the operand tile, so that reads and writes are
    // free of bank conflicts as they come. The converters share the issue slots of the
    // softmax warps, whose latency sets the pace: every instruction here counts.
    constexpr int kGroups = D / 8, kRowsIter = 32 / kGroups, kIters = 32 / kRowsIter;
    const int cw = warp - kConvWarp;
    const int lo = w.lo, n_kv = w.hi - w.lo, L_seq = w.span.L;
    const int grp = lane % kGroups, sub = lane / kGroups;
    const int row0 = cw * 32 + sub;
    // swizzled column of this lane's write in iteration it: a function of it % kTurns
    constexpr int kTurns = 8 / kRowsIter;
    int column[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
      column[k] = (grp >> 3) * L::kChunk + row0 * 128 + (((grp & 7) ^ ((sub + k * kRowsIter) & 7)) << 4);
    const int depth = w.dual ? S::kCodeStagesDual : S::kCodeStages;
    bool live = true;
    int e_ref = 0, e_k = 0, e_v = 0, cs = -1, skip = skipped();
    uint32_t code_parity = 1;
    for (int u = 0; u < 2 * n_kv; ++u) {
      if (++cs == depth) cs = 0;
      if (cs == 0) code_parity ^= 1;
      const int s = u % kStages, jj = u >> 1;
      const bool is_v = u & 1;
      if (live)
        live = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->code_full[cs]), code_parity, wc));
      if (u == 2) skip = 0;
      const int valid = imin(BN, L_seq - (lo + jj) * BN);
      const bool partial = valid < BN || skip > 0;
      const uint8_t* ex = smem + L::kExp + (jj % kInfo) * BN * 2;
      if (live && !is_v) {  // the tile's exponents: lane reads rows 4 lane .. + 3 (K low byte)
        uint2 x = *reinterpret_cast<const uint2*>(ex + lane * 8);
        if (partial) {  // (skip is a multiple of 8: a lane's rows are in or out together)
          const int in = 4 * lane < skip ? 0 : valid - 4 * lane;
          x.x &= in >= 2 ? 0xFFFFFFFFu : in == 1 ? 0xFFFFu : 0u;
          x.y &= in >= 4 ? 0xFFFFFFFFu : in == 3 ? 0xFFFFu : 0u;
        }
        constexpr uint32_t kLow = 0x00FF00FFu;
        const uint32_t mk = __vmaxu2(x.x & kLow, x.y & kLow);
        const uint32_t mv = __vmaxu2((x.x >> 8) & kLow, (x.y >> 8) & kLow);
        e_k = (int)__reduce_max_sync(0xffffffffu, max(mk & 255u, mk >> 16));
        e_v = (int)__reduce_max_sync(0xffffffffu, max(mv & 255u, mv >> 16));
        e_ref = imax(e_ref, e_v);
        e_v = imax(e_v, e_ref - kMaxDown);
      }
      if (live)
        live = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->kv_empty[s]),
                                                 ((u / kStages) & 1) ^ 1, wc));
      if (!live) {
        nb_sync(kNbKv + s, S::kNbKvCount);
        continue;
      }
      if (!is_v && cw == 0 && lane == 0) {
        bars->info[jj % kInfo] = make_int4(e_k, e_v, e_ref, 0);
        mbar_arrive(smem_u32(&bars->info_full[jj % kInfo]));
      }
      // 2^(e_j - E) of row cw * 32 + lane as an fp16 pair (0 below fp16's range)
      const int e_row = ex[(cw * 32 + lane) * 2 + is_v];
      const float ff = __uint_as_float((uint32_t)imax(127 - (is_v ? e_v : e_k) + e_row, 0) << 23);
      const uint32_t factor = pack_f16x2(ff, ff);
      const uint8_t* src = code_tile(cs) + row0 * D + grp * 8;
      uint8_t* dst = smem + L::kRing + s * L::kTile;
#pragma unroll
      for (int it0 = 0; it0 < kIters; it0 += 8) {
        uint2 c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          c[q] = *reinterpret_cast<const uint2*>(src + (it0 + q) * kRowsIter * D);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int it = it0 + q;
          const uint32_t f = __shfl_sync(0xffffffffu, factor, it * kRowsIter + sub);
          uint32_t h[4];
          decode4(c[q].x, h[0], h[1]);
          decode4(c[q].y, h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + column[it % kTurns] + it * kRowsIter * 128) =
              make_uint4(mul_f16x2(h[0], f), mul_f16x2(h[1], f), mul_f16x2(h[2], f), mul_f16x2(h[3], f));
        }
      }
      if (partial) {  // the other rows hold anything, NaN codes included: clear
        __syncwarp();
        for (int e = lane; e < 32 * 8 * L::kSlabs; e += 32) {
          const int slab = e / 256, row = cw * 32 + (e % 256) / 8;
          if (row < skip || row >= valid)
            *reinterpret_cast<uint4*>(smem + L::kRing + s * L::kTile + slab * L::kChunk + row * 128 +
                                      (e % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->code_empty[cs]));
      nb_arrive(kNbKv + s, S::kNbKvCount);
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<S::kRegsOther>();
    if (warp == kLoadKWarp || warp == kLoadVWarp) {
      // ------------------------------------------------------------ loaders
      // One warp for K, one for V (small pages: the copies of one tile take a warp hundreds
      // of clocks to issue). Lane q fetches the q-th page piece of a tile: TMA boxes (bf16) or
      // a bulk copy (codes). K tiles take the even stages of the ring, V tiles the odd ones.
      const bool is_v = warp == kLoadVWarp;
      const int R = piece_keys(), pieces = BN / R;
      const int lo = w.lo, hi = w.hi, n_kv = hi - lo, k_lo = w.k_lo;
      auto rows_of = [&](int j) -> int {  // cache row of this lane's piece, or -1
        const int key = j * BN + lane * R;
        if (j >= hi || lane >= pieces || key >= w.span.L || key + R <= k_lo) return -1;
        const long long r = cache_row(p, w.b, key, w.hk);
        if (r < 0) atomicOr(p.status, DEV_BAD_INPUT);
        return (int)r;
      };
      const int depth = !kE4m3 ? kStages : w.dual ? S::kCodeStagesDual : S::kCodeStages;
      const uint32_t full = smem_u32(kE4m3 ? bars->code_full : bars->kv_full);
      const uint32_t empty = smem_u32(kE4m3 ? bars->code_empty : bars->kv_empty);
      int row = rows_of(lo), next = rows_of(lo + 1);
      bool live = true;
      int issued = 0, s = is_v - 2;
      uint32_t parity = 0;  // of the stage's last release; the first turn finds it released
      for (int jj = 0; jj < n_kv && live; ++jj) {
        s += 2;
        if (s >= depth) s -= depth;
        if (s < 2) parity ^= 1;
        live = __all_sync(0xffffffffu, mbar_wait(empty + s * 8, parity, wc));
        if (!live) break;
        const uint32_t bar = full + s * 8;
        const uint32_t n = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0));
        if (lane == 0)
          mbar_arrive_expect_tx(bar, kE4m3 ? n * R * (D + (is_v ? 0 : 2)) : n * R * D * 2);
        __syncwarp();
        if (row >= 0) {
          if constexpr (kE4m3) {
            const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache);
            bulk_load(smem_u32(code_tile(s)) + lane * R * D, src + (size_t)row * D, R * D, bar);
            if (!is_v)  // the exponents of K and V come with K
              bulk_load(smem_u32(smem + L::kExp + (jj % kInfo) * BN * 2) + lane * R * 2,
                        p.kv_exp + (size_t)row * 2, R * 2, bar);
          } else {
#pragma unroll
            for (int c = 0; c < L::kSlabs; ++c)
              tma_load_3d(smem_u32(smem + L::kRing + s * L::kTile + c * L::kChunk) + lane * R * 128,
                          is_v ? &tm_v : &tm_k, bar, c * 64, row, 0);
          }
        }
        ++issued;
        row = next;
        next = rows_of(lo + jj + 2);
      }
      // Do not leave while copies into this CTA's shared memory are in flight.
      for (int jj = imax(0, issued - depth / 2); jj < issued; ++jj) {
        const int u = 2 * jj + is_v;
        drain_wait(full + (u % depth) * 8, (u / depth) & 1);
      }
    } else if (!kE4m3 && warp == kRelayWarp) {
      // ------------------------------------------------------------ relay (bf16)
      // After a ring use's bytes have landed (and the V rows behind the sequence or not loaded
      // are cleared), arrive on its named barrier for the MMA warp. After an abort, rendezvous.
      bool live = true;
      const int lo = w.lo, n_kv = w.hi - lo;
      int skip = skipped();
      for (int u = 0; u < 2 * n_kv; ++u) {
        const int s = u % kStages;
        if (live)
          live = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->kv_full[s]), (u / kStages) & 1, wc));
        if (u == 2) skip = 0;
        const int valid = w.span.L - (lo + (u >> 1)) * BN;
        if (live && (u & 1) && (valid < BN || skip > 0)) {
          for (int e = lane; e < BN * 8 * L::kSlabs; e += 32) {
            const int slab = e / (BN * 8), row = e / 8 % BN;
            if (row < skip || row >= valid)
              *reinterpret_cast<uint4*>(smem + L::kRing + s * L::kTile + slab * L::kChunk +
                                        row * 128 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (live) nb_arrive(kNbKv + s, S::kNbKvCount);
        else nb_sync(kNbKv + s, S::kNbKvCount);
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      // As in the forward kernel: the whole warp walks the schedule and waits on named
      // barriers; one elected lane issues. If Q never arrives it issues nothing.
      constexpr uint32_t idS = kE4m3 ? idesc_f16_f32(BM, BN, false) : idesc_bf16_f32(BM, BN, false, false);
      constexpr uint32_t idO = kE4m3 ? idesc_f16_f32(BM, D, true) : idesc_bf16_f32(BM, D, false, true);
      const uint32_t q_base = smem_u32(smem + L::kQ);
      const uint32_t ring = smem_u32(smem + L::kRing);
      int np[kQTiles] = {0, 0};
      const int lo = w.lo, n_kv = w.hi - lo;
      const bool dual = w.dual;
      const int t_lo[kQTiles] = {w.tk[0].lo, w.tk[1].lo}, t_hi[kQTiles] = {w.tk[0].hi, w.tk[1].hi};
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->q_full), 0, wc));
      tc_fence_after_sync();
      const bool issuer = elect_one();
      auto commit = [&](uint64_t* bar) {
        if (ok) mma_commit_if(issuer, smem_u32(bar));
      };
      auto sync_stage = [&](int u) {
        nb_sync(kNbKv + u % kStages, S::kNbKvCount);
        tc_fence_after_sync();
      };
      auto issue_s = [&](int t, int u) {
        if (!ok) return;
        const uint64_t dq = smem_desc_sw128(q_base + (dual ? 0 : t * L::kTile), 16, 1024);
        const uint64_t dk = smem_desc_sw128(ring + (u % kStages) * L::kTile, 16, 1024);
        const uint32_t col = t == 0 ? L::kColS0 : L::kColS1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * L::kChunk + (kk & 3) * 32) >> 4;
          mma_ss_if(issuer, tmem + col, dq + off, dk + off, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit_if(issuer, smem_u32(&bars->s_full[t]));
      };
      // O_t += P_t V, each part as soon as its P is there (add: O_t holds earlier products).
      auto issue_pv = [&](int t, int u, bool add) {
        const uint32_t colS = t == 0 ? L::kColS0 : L::kColS1;
        const uint32_t colO = t == 0 ? L::kColO0 : L::kColO1;
        const uint64_t dv = smem_desc_sw128(ring + (u % kStages) * L::kTile, L::kChunk, 1024);
#pragma unroll
        for (int part = 0; part < S::kPParts; ++part) {
          nb_sync(kNbP + 2 * t + part, kNbPCount);
          tc_fence_after_sync();
          if (!ok) continue;
          constexpr int kSteps = BN / 16 / S::kPParts;
#pragma unroll
          for (int kk = part * kSteps; kk < (part + 1) * kSteps; ++kk)
            mma_ts_if(issuer, tmem + colO, tmem + colS + kk * 8, dv + ((kk * 16 * 128) >> 4), idO,
                      (add || kk > 0) ? 1u : 0u);
        }
      };
      sync_stage(0);
      if (dual) {  // key tile jj belongs to stream jj & 1; S runs one tile ahead
        issue_s(0, 0);
        commit(&bars->kv_empty[0]);
        for (int jj = 0; jj < n_kv; ++jj) {
          const int t = jj & 1, uv = 2 * jj + 1, uk = 2 * jj + 2;
          if (jj + 1 < n_kv) {
            sync_stage(uk);
            issue_s(t ^ 1, uk);
            commit(&bars->kv_empty[uk % kStages]);
          }
          sync_stage(uv);
          issue_pv(t, uv, jj > 1);
          commit(&bars->kv_empty[uv % kStages]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < kQTiles; ++t)
          if (lo >= t_lo[t] && lo < t_hi[t]) issue_s(t, 0);
        commit(&bars->kv_empty[0]);
        for (int jj = 0; jj < n_kv; ++jj) {
          const int j = lo + jj;
          const int uv = 2 * jj + 1, uk = 2 * jj + 2;
          const bool next = jj + 1 < n_kv;
          sync_stage(uv);
#pragma unroll
          for (int t = 0; t < kQTiles; ++t) {
            if (j >= t_lo[t] && j < t_hi[t]) {
              issue_pv(t, uv, np[t] > 0);
              ++np[t];
            }
            if (next) {
              if (t == 0) sync_stage(uk);
              if (j + 1 >= t_lo[t] && j + 1 < t_hi[t]) issue_s(t, uk);
            }
          }
          commit(&bars->kv_empty[uv % kStages]);
          if (next) commit(&bars->kv_empty[uk % kStages]);
        }
      }
#pragma unroll
      for (int t = 0; t < kQTiles; ++t) commit(&bars->o_full[t]);
    }
  } else {
    setmaxnreg_inc<S::kRegsSoftmax>();
    // ------------------------------------------------------------ softmax warpgroups
    const int t = wt;
    const int row = (warp & 3) * 32 + lane;     // TMEM lane = row in the tile
    const int r = wrow + lane;                  // row in the unit
    const bool has_row = r < w.rows;
    float row_scale = 1.f;  // e4m3: undoes the power of two that this thread's row was scaled by
    {
      // This warp's 32 Q rows into swizzled shared memory (rows past the end: zeros). e4m3:
      // scaled by a power of two to fp16.
      const int piece = lane % kPer;
#pragma unroll
      for (int it = 0; it < kQIters; ++it) {
        if constexpr (kE4m3) {
          uint32_t u[4] = {qv[it].x, qv[it].y, qv[it].z, qv[it].w};
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(u[e] & 0x7FFFu, (u[e] >> 16) & 0x7FFFu));
#pragma unroll
          for (int off = kPer / 2; off > 0; off >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
          const int x = imax((int)(top >> 7) - 127, -112);
          const float up = __uint_as_float((uint32_t)(14 - x + 127) << 23);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            u[e] = pack_f16x2(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xFFFF0000u) * up);
          qv[it] = make_uint4(u[0], u[1], u[2], u[3]);
          const int xl = __shfl_sync(0xffffffffu, x, lane % kRowsPerIter * kPer);
          if (lane / kRowsPerIter == it) row_scale = __uint_as_float((uint32_t)(xl - 14 + 127) << 23);
        }
        const int rt = (warp & 3) * 32 + it * kRowsPerIter + lane / kPer;
        if (t == 0 || !w.dual)  // (a dual unit's streams share the tile)
          *reinterpret_cast<uint4*>(smem + L::kQ + t * L::kTile + (piece >> 3) * L::kChunk + rt * 128 +
                                    (((piece & 7) ^ (rt & 7)) << 4)) = qv[it];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
    }
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + (t == 0 ? L::kColS0 : L::kColS1);
    const uint32_t tO = tmem + lane_base + (t == 0 ? L::kColO0 : L::kColO1);
    const Row me = row_of(imin(r, w.rows - 1));
    const int pos = w.span.L - w.span.n + me.i;
    int row_lo, row_hi;  // allowed keys of this row in this chunk
    decode_row_keys(a.mask_kind, a.window, w.span.L, w.span.n, me.i, row_lo, row_hi);
    row_lo = imax(row_lo, w.c0);
    row_hi = imin(row_hi, w.c1);
    const bool dual = w.dual;
    const TileKeys tk = w.tk[dual ? 0 : t];
    const int lo = w.lo;
    const float slope = kAlibi ? alibi_slope(me.h, a.Hq) : 0.f;
    const float unit = kSoftcap ? 1.0f / a.softcap : kPagedLog2e;
    const float k1 = a.scale * unit * row_scale;
    const float kb = slope * unit;
    const float capA = kSoftcap ? a.softcap * kPagedLog2e : 0.f;
    const bool raw_ok = !kAlibi && !kSoftcap && a.scale > 0.f;
    float m_run = -INFINITY, l_run = 0.f;
    int n = 0, e_ref = 0;
    bool live = true;
    for (int j = tk.lo + (dual ? t : 0); j < tk.hi; j += dual ? 2 : 1, ++n) {
      int4 info = make_int4(127, 127, 127, 0);
      if (kE4m3 && n > 0 && live) {
        // The tile's scales are there long before its scores; having seen tile j - 1's, this
        // thread cannot be a whole turn of the slots behind, which the parity would not show.
        const int jj = j - lo;
        live = mbar_wait(smem_u32(&bars->info_full[jj % kInfo]), (jj / kInfo) & 1, wc);
        info = bars->info[jj % kInfo];
      }
      live = __all_sync(0xffffffffu, live && mbar_wait(smem_u32(&bars->s_full[t]), n & 1, wc));
      if (kE4m3 && n == 0 && live) {  // the first tile: its scores show that the turn is right
        const int jj = j - lo;
        live = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->info_full[jj % kInfo]), (jj / kInfo) & 1, wc));
        info = bars->info[jj % kInfo];
      }
      if (!live) {  // aborted: keep the barrier schedule with the MMA warp, do nothing else
        for (int part = 0; part < S::kPParts; ++part) nb_sync(kNbP + 2 * t + part, kNbPCount);
        continue;
      }
      tc_fence_after_sync();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, x[c]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) reg_fence32(x[c]);
      const int k0 = j * BN;
      const float k1j = kE4m3 ? k1 * exp_byte_scale((uint32_t)info.x) : k1;
      const bool masked = k0 < tk.full_lo || k0 + BN > tk.full_hi;  // warp-uniform
      const bool fast = raw_ok && !masked;
      float mx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx[e] = -INFINITY;
      if (fast) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) mx[e & 7] = fmaxf(mx[e & 7], __uint_as_float(x[c][e]));
      } else {
        const int c_lo = row_lo - k0, c_hi = row_hi - k0;  // allowed columns [c_lo, c_hi)
        const float base = kAlibi ? (float)(k0 - pos) * kb : 0.f;
        const uint64_t k1j2 = f32x2(k1j, k1j);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int col = c * 32 + e;
            const uint64_t x2 = f32x2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
            uint64_t s2 = kAlibi ? fma_f32x2(x2, k1j2,
                                             f32x2(fmaf((float)col, kb, base),
                                                   fmaf((float)(col + 1), kb, base)))
                                 : mul_f32x2(x2, k1j2);
            float v0, v1;
            f32x2_split(s2, v0, v1);
            if (kSoftcap) {
              v0 = tanh_approx(v0);
              v1 = tanh_approx(v1);
            }
            if (masked) {
              v0 = (col >= c_lo && col < c_hi) ? v0 : -INFINITY;
              v1 = (col + 1 >= c_lo && col + 1 < c_hi) ? v1 : -INFINITY;
            }
            mx[e & 7] = fmaxf(mx[e & 7], v0);
            mx[(e + 1) & 7] = fmaxf(mx[(e + 1) & 7], v1);
            x[c][e] = __float_as_uint(v0);
            x[c][e + 1] = __float_as_uint(v1);
          }
      }
      float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                       fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
      if (fast) mt *= k1j;
      else if (kSoftcap) mt *= capA;
      const float m_new = fmaxf(m_run, mt);
      const bool e_grow = kE4m3 && n > 0 && info.z > e_ref;
      const bool warp_grow = __any_sync(0xffffffffu, m_new > m_run + S::kLag || e_grow);
      float corr = 1.f;
      if (warp_grow) {
        corr = m_new == -INFINITY ? 1.f : ex2_approx(m_run - m_new);
        m_run = m_new;
        l_run *= corr;
        if (kE4m3) {  // O also moves to the new reference exponent
          const int up = info.z - e_ref;
          corr = up > 126 ? 0.f : corr * __uint_as_float((uint32_t)(127 - up) << 23);
        }
      }
      if (kE4m3) e_ref = info.z;
      float neg_m = m_run == -INFINITY ? 0.f : -m_run;
      if (kE4m3) neg_m += kPOffset + (float)(info.y - info.z);
      const float mul = fast ? k1j : (kSoftcap ? capA : 1.f);
      uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
      const uint64_t mul2 = f32x2(mul, mul), negm2 = f32x2(neg_m, neg_m), one2 = f32x2(1.f, 1.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t ph[8];
#pragma unroll
          for (int e8 = 0; e8 < 8; ++e8) {
            const int e = hf * 8 + e8;
            float a0, a1;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])),
                                  mul2, negm2), a0, a1);
            const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
            acc2[e & 3] = fma_f32x2(f32x2(p0, p1), one2, acc2[e & 3]);
            ph[e8] = kE4m3 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
          tmem_st8(tS + c * 16 + hf * 8, ph);
        }
        if ((c + 1) % (4 / S::kPParts) == 0) {  // a part is in: its products may start
          if (c + 1 == 4 / S::kPParts && warp_grow && n > 0) {
            if constexpr (S::kPParts == 1) {
#pragma unroll
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(tO + q * 32, o);
                tmem_wait_ld();
                reg_fence32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st32(tO + q * 32, o);
              }
            } else {  // 16 columns at a time: 64 scores are still in registers
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(tO + q * 16, o);
                tmem_wait_ld();
                reg_fence16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st16(tO + q * 16, o);
              }
            }
          }
          tmem_wait_st();
          tc_fence_before_sync();
          nb_arrive(kNbP + 2 * t + c * S::kPParts / 4, kNbPCount);
        }
      }
      float acc[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) f32x2_split(acc2[e], acc[2 * e], acc[2 * e + 1]);
      const float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
      // the row sum keeps the plain weights (0 <= E_ref - E_V <= kMaxDown)
      l_run = kE4m3 ? fmaf(sum, __uint_as_float((uint32_t)(127 + info.z - info.y) << 23), l_run) : l_run + sum;
    }
    // ---------------------------------------------------------- epilogue
    grid_dependents_launch();
    // Every tile waits for the CTA's last MMA: the staging below writes over Q.
    const bool mma_done = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->o_full[t]), 0, wc));
    const bool have_o = n > 0 && mma_done;
    tc_fence_after_sync();
    const float vs = kE4m3 ? exp_byte_scale((uint32_t)e_ref) : 1.f;
    // A dual unit: the second warpgroup leaves its O rows, their maxima, sums and scale in the
    // ring, which no one uses any more; the first one merges. The scales come last: V may lie
    // near the top of fp32's range, and O carries 2^11 and the row sum until it is divided.
    float* other = reinterpret_cast<float*>(smem + L::kRing);   // [row][D], pieces swizzled
    float* other_ml = other + BM * D;                           // [row][4]
    static_assert(BM * (D + 4) * 4 <= S::kStages * L::kTile, "merge space");
    float f0 = 1.f, f1 = 0.f, vs1 = 1.f;
    if (dual) {
      if (t == 1) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (have_o) {
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld();
            reg_fence32(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(other + row * D + (((c * 8 + e) ^ (row & (D / 4 - 1))) << 2)) =
                make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
        *reinterpret_cast<float4*>(other_ml + row * 4) = make_float4(m_run, l_run, vs, 0.f);
      }
      nb_sync(kNbDual, 256);
      if (t == 0) {
        const float4 ml = *reinterpret_cast<const float4*>(other_ml + row * 4);
        vs1 = ml.z;
        const float M = fmaxf(m_run, ml.x);
        f0 = m_run == -INFINITY ? 0.f : ex2_approx(m_run - M);
        f1 = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
        l_run = l_run * f0 + ml.y * f1;
        m_run = M;
      }
    }
    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // (a NaN sum makes the row NaN)
    f0 *= inv;
    f1 *= inv;
    const float l2 = l_run == 0.f ? -INFINITY : m_run + log2f(l_run) - (kE4m3 ? kPOffset : 0.f);
    const bool mine = !dual || t == 0;  // warp-uniform: this warpgroup writes the rows
    // 32 columns of the finished row
    auto load_o = [&](int c, float (&v)[32]) {
      uint32_t o[32];
      if (have_o) {
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld();
        reg_fence32(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * f0 * vs;
      if (dual && f1 > 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 x = *reinterpret_cast<const float4*>(other + row * D + (((c * 8 + e) ^ (row & (D / 4 - 1))) << 2));
          v[4 * e] = fmaf(x.x * f1, vs1, v[4 * e]);
          v[4 * e + 1] = fmaf(x.y * f1, vs1, v[4 * e + 1]);
          v[4 * e + 2] = fmaf(x.z * f1, vs1, v[4 * e + 2]);
          v[4 * e + 3] = fmaf(x.w * f1, vs1, v[4 * e + 3]);
        }
      }
    };
    if (mine && a.n_chunks > 1) {
      const long long part = ((long long)w.cc * p.T + me.t) * a.Hq + me.h;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        load_o(c, v);
        if (!has_row) continue;
        float4* dst = reinterpret_cast<float4*>(a.part_o + part * D + c * 32);
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
      }
      if (has_row) a.part_lse[part] = l2;
    } else if (mine) {
      uint8_t* otile = smem + t * L::kTile;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float v[32];
        load_o(c, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int gc = c * 4 + e;  // 16-byte piece of the row
          *reinterpret_cast<uint4*>(otile + (gc >> 3) * L::kChunk + row * 128 + (((gc & 7) ^ (row & 7)) << 4)) =
              make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                         pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
        }
      }
      __syncwarp();
      const int gc = lane % kPer;
#pragma unroll 4
      for (int k = 0; k < kQIters; ++k) {
        const int rt = (warp & 3) * 32 + k * kRowsPerIter + lane / kPer;
        const uint4 v = *reinterpret_cast<const uint4*>(otile + (gc >> 3) * L::kChunk + rt * 128 +
                                                       (((gc & 7) ^ (rt & 7)) << 4));
        const int ru = (dual ? 0 : t * BM) + rt;
        if (ru < w.rows) reinterpret_cast<uint4*>(o_row(row_of(ru)))[gc] = v;
      }
      if (has_row) *lse_row(me) = l2 * kPagedLn2;
    }
  }
  __syncwarp();

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <int D, bool kAlibi, bool kSoftcap, bool kE4m3>
cudaError_t launch_variant(const PagedAttention& a, const PagedMaps& maps, unsigned grid,
                           cudaStream_t st) {
  using S = Shape<kE4m3>;
  auto kern = paged_tiles_kernel<D, kAlibi, kSoftcap, kE4m3>;
  const int smem = Layout<D, kE4m3>::kAlloc;
  // The register split of setmaxnreg waits for ever unless the launch brings kRegsLaunch
  // registers a thread: refuse to launch a build in which it does not.
  static const bool regs_ok = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kern) == cudaSuccess && attr.numRegs >= S::kRegsLaunch;
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  kern<<<grid, S::kThreads, smem, st>>>(maps.k, maps.v, a);
  return cudaGetLastError();
}

template <bool kE4m3>
cudaError_t launch_tiles(const PagedAttention& a, const PagedMaps& maps, cudaStream_t st) {
  const PagedProblem& p = a.p;
  // Row units: at most T G / 256 full ones and one more per sequence.
  const long long per_seq = ((long long)p.max_new * a.G + kUnitRows - 1) / kUnitRows;
  const long long units = imin64((long long)p.T * a.G / kUnitRows + p.B, per_seq * p.B);
  // (one CTA at least: it reports chunks that are longer than a max_new of 0)
  const long long grid = units * p.Hkv * a.n_chunks > 0 ? units * p.Hkv * a.n_chunks : 1;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)grid;
  const bool al = a.score_kind & ATTN_SCORE_ALIBI, sc = a.score_kind & ATTN_SCORE_SOFTCAP;
  if (p.d == 64) {
    if (al && sc) return launch_variant<64, true, true, kE4m3>(a, maps, g, st);
    if (al) return launch_variant<64, true, false, kE4m3>(a, maps, g, st);
    if (sc) return launch_variant<64, false, true, kE4m3>(a, maps, g, st);
    return launch_variant<64, false, false, kE4m3>(a, maps, g, st);
  }
  if (al && sc) return launch_variant<128, true, true, kE4m3>(a, maps, g, st);
  if (al) return launch_variant<128, true, false, kE4m3>(a, maps, g, st);
  if (sc) return launch_variant<128, false, true, kE4m3>(a, maps, g, st);
  return launch_variant<128, false, false, kE4m3>(a, maps, g, st);
}

}  // namespace pt
}  // namespace attn
