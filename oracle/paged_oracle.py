"""Float64 CPU oracle of the paged cache's operators: the e4m3 cache format, writing and
reading tokens, and attention of ragged chunks of new tokens over the cache.

TEST INFRASTRUCTURE ONLY, like ``attention_oracle``: the library never imports it.

Format: a code's value is its e4m3 value (sign, 4 exponent bits with bias 7, 3 mantissa
bits; 0x7F and 0xFF are NaN) times 2^(exp - 127), one exponent byte per token, kv head and
tensor (kv_exp[..., 0] for K, [..., 1] for V). A row is written under the smallest e in
[-127, 127] with amax <= 448 * 2^e, amax its largest finite magnitude (e = -127 for zeros);
codes are the nearest e4m3 values, ties to even; NaN and infinities become NaN.

Chunk attention is ``decode_oracle``'s with ragged packed rows: row i of sequence b's n_b
new tokens sits at position seq_lens[b] - n_b + i.
"""
from __future__ import annotations

import numpy as np

from . import attention_oracle as ref


def e4m3_values() -> np.ndarray:
    """The 256 code values."""
    c = np.arange(256)
    s = np.where(c & 128, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return s * v


def encode(x: np.ndarray):
    """x float64 [..., d] -> (codes uint8 [..., d], exponent bytes uint8 [...])."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = finite.max(axis=-1)
    e = np.full(amax.shape, -127, dtype=np.int64)
    for k in range(-127, 128):  # the definition, by counting
        e = np.where(amax > 448.0 * 2.0 ** k, min(k + 1, 127), e)
    y = x / 2.0 ** e[..., None]
    table = e4m3_values()
    pos = table[:127]                                     # 0 .. 448 ascending
    mag = np.where(np.isfinite(y), np.abs(y), 0.0)
    hi = np.clip(np.searchsorted(pos, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(mag == 0.0, 0, code)
    code = code | np.where(np.signbit(y), 128, 0)
    code = np.where(np.isfinite(x), code, 127)
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def decode(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    return e4m3_values()[codes] * 2.0 ** (exps.astype(np.float64) - 127.0)[..., None]


def cache_rows(page_table_row, page_size: int, lo: int, hi: int):
    """(pages, slots) of tokens lo .. hi - 1 of one sequence."""
    t = np.arange(lo, hi)
    return np.asarray(page_table_row, dtype=np.int64)[t // page_size], t % page_size


def sequence(k_cache, v_cache, kv_exp, page_table_row, lo: int, hi: int):
    """K and V of tokens lo .. hi - 1 of one sequence, float64 [hi - lo, Hkv, d]."""
    ps = k_cache.shape[2]
    pages, slots = cache_rows(page_table_row, ps, lo, hi)
    out = []
    for i, c in enumerate((k_cache, v_cache)):
        rows = ref._f64(c)[pages, :, slots] if kv_exp is None else \
            decode(np.asarray(c)[pages, :, slots], np.asarray(kv_exp)[pages, :, slots, i])
        out.append(rows)
    return out


def chunk_forward(q, k_cache, v_cache, kv_exp, page_table, offsets, seq_lens, scale,
                  mask_kind=0, window=0, score_kind=0, softcap=0.0, rows=None):
    """q [T, Hq, d] -> (O [T, Hq, d], LSE [T, Hq], A [T, Hq, d]) float64, A = sum_j P |V|, the
    magnitude of the terms summed into O. Rows of no sequence are NaN; ``rows`` limits the
    packed rows computed."""
    q = ref._f64(q)
    T, Hq, d = q.shape
    G = Hq // k_cache.shape[1]
    out, mag = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse = np.full((T, Hq), np.nan)
    offs, lens = np.asarray(offsets), np.asarray(seq_lens)
    for b in range(len(lens)):
        L = int(lens[b])
        t = np.arange(int(offs[b]), int(offs[b + 1]))
        pos = L - len(t) + np.arange(len(t))
        if rows is not None:
            keep = np.isin(t, rows)
            t, pos = t[keep], pos[keep]
        if len(t) == 0:
            continue
        K, V = sequence(k_cache, v_cache, kv_exp, page_table[b], 0, L)
        cols = np.arange(L)
        ok = ref.allowed(mask_kind, pos, cols, window) if L else np.zeros((len(t), 0), bool)
        for h in range(Hq):
            s = float(scale) * (q[t, h] @ K[:, h // G].T)
            if score_kind & ref.SCORE_ALIBI:
                s = s - ref.alibi_slope(h, Hq) * (pos[:, None] - cols[None, :])
            if score_kind & ref.SCORE_SOFTCAP:
                s = softcap * np.tanh(s / softcap)
            s = np.where(ok, s, -np.inf)
            m = s.max(axis=1, initial=-np.inf)
            live = m > -np.inf
            e = np.where(ok, np.exp(s - np.where(live, m, 0.0)[:, None]), 0.0)
            l = e.sum(axis=1)
            p = e / np.where(live, l, 1.0)[:, None]
            out[t, h] = p @ V[:, h // G]
            mag[t, h] = p @ np.abs(V[:, h // G])
            with np.errstate(divide="ignore"):
                lse[t, h] = np.where(live, np.where(live, m, 0.0) + np.log(l), -np.inf)
    return out, lse, mag
