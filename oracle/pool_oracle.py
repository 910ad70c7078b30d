"""Plain CPU definitions of the operators around the paged cache: pages forked, resized,
compacted and copied, and the verification of drafted tokens.

TEST INFRASTRUCTURE ONLY, like ``attention_oracle``: the library never imports it. State is a
page table (list of rows), lengths and counts of holders, changed by small loops that follow the
statements of include/attn.h one by one; caches are numpy arrays [pages, Hkv, page_size, ...].
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def pages_of(tokens: int, page_size: int) -> int:
    return -(-tokens // page_size)


def fork(table, lens, refs, parents, page_size):
    """(table, lens, refs) after row i took what row parents[i] held."""
    old, old_lens = [list(r) for r in table], list(lens)
    table, refs = [list(r) for r in table], list(refs)
    new_lens = [0 if p < 0 else old_lens[p] for p in parents]
    for b, p in enumerate(parents):
        before, after = pages_of(old_lens[b], page_size), pages_of(new_lens[b], page_size)
        for e in old[b][:before]:
            if e >= 0:
                refs[e] -= 1
        for i in range(max(before, after)):
            table[b][i] = old[p][i] if i < after else -1
            if i < after and old[p][i] >= 0:
                refs[old[p][i]] += 1
    return table, new_lens, refs


def resize(table, lens, refs, new_lens, page_size, window=0):
    """(table, lens, refs, missing, copies): copies are (from, to, tokens)."""
    start = [list(r) for r in table], list(lens), list(refs)
    table, refs = [list(r) for r in table], list(refs)
    for row, L, N in zip(table, lens, new_lens):
        gone = list(range(pages_of(N, page_size), pages_of(L, page_size)))
        if window > 0:
            i = (min(L, N) - window + 1) // page_size - 1     # the last page wholly below
            while i >= 0 and row[i] >= 0:
                gone.append(i)
                i -= 1
        for i in gone:
            if row[i] >= 0:
                refs[row[i]] -= 1
            row[i] = -1
    wants = [[] for _ in table]
    for b, (row, L, N) in enumerate(zip(table, lens, new_lens)):
        if N > L and L % page_size:
            e = row[L // page_size]
            writers = [x for x in range(len(table)) if new_lens[x] > lens[x] and
                       lens[x] % page_size and table[x][lens[x] // page_size] == e]
            if refs[e] > len(writers) or (refs[e] > 1 and b != writers[0]):
                wants[b].append(L // page_size)
        wants[b] += range(pages_of(L, page_size), pages_of(N, page_size))
    free = [p for p, r in enumerate(refs) if r == 0]
    need = sum(len(w) for w in wants)
    if need > len(free):
        return (*start, need - len(free), [])
    copies = []
    for b, row in enumerate(table):
        for i in wants[b]:
            page = free.pop(0)
            if i * page_size < lens[b]:
                copies.append((row[i], page, lens[b] % page_size))
            row[i] = page
            refs[page] = 1
    for src, _, _ in copies:
        refs[src] -= 1
    return table, list(new_lens), refs, 0, copies


def compact(table, lens, refs, page_size):
    """(table, refs, used, page_map, moves): moves are (from, to)."""
    table, refs = [list(r) for r in table], list(refs)
    used = [p for p, r in enumerate(refs) if r != 0]
    high = sorted((p for p in used if p >= len(used)), reverse=True)
    low = [p for p in range(len(used)) if refs[p] == 0]
    page_map = [p if r != 0 else -1 for p, r in enumerate(refs)]
    for src, dst in zip(high, low):
        page_map[src], refs[dst], refs[src] = dst, refs[src], 0
    for row, L in zip(table, lens):
        for i in range(pages_of(L, page_size)):
            if row[i] >= 0:
                row[i] = page_map[row[i]]
    return table, refs, len(used), page_map, list(zip(high, low))


def copy_pages(cache, to, moves):
    """Copies (from, to) or (from, to, tokens) of each array of `cache` into that of `to`."""
    for x, y in zip(cache, to):
        if x is None:
            continue
        before = x.copy()
        for m in moves:
            n = m[2] if len(m) > 2 else x.shape[2]
            y[m[1], :, :n] = before[m[0], :, :n]


def _weights(p, q=None):
    """Positive finite max(p - q, 0) as exact fractions."""
    out = []
    for x in range(len(p)):
        a, b = float(p[x]), 0.0 if q is None else float(q[x])
        ok = np.isfinite(a) and np.isfinite(b) and a > b
        out.append(Fraction(a) - Fraction(b) if ok else Fraction(0))
    return out


def verify(target, draft, tokens, offsets, accept_u, sample_u):
    """(accepted, next_tokens), every comparison in exact arithmetic."""
    accepted, nxt = [], []
    V = target.shape[1]
    for b in range(len(offsets) - 1):
        r0, r1 = int(offsets[b]), int(offsets[b + 1])
        if r0 == r1:
            accepted.append(0), nxt.append(-1)
            continue
        w = None
        t = r0
        while t < r1 - 1:
            x = int(tokens[t + 1])
            one = draft is None
            if not (0 <= x < V and np.isfinite(accept_u[t]) and np.isfinite(float(target[t, x])) and
                    float(target[t, x]) > 0 and (one or np.isfinite(float(draft[t, x]))) and
                    Fraction(float(accept_u[t])) * (1 if one else Fraction(float(draft[t, x])))
                    < Fraction(float(target[t, x]))):
                q = np.zeros(V) if one else draft[t]
                w = _weights(target[t], q)
                if one and 0 <= x < V:
                    w[x] = Fraction(0)
                if not sum(w):
                    w = _weights(target[t])
                break
            t += 1
        if w is None:
            w = _weights(target[t])
        total, run, token, last = sum(w), Fraction(0), -1, -1
        for x in range(V):
            run += w[x]
            if w[x]:
                last = x
            if run > Fraction(float(sample_u[b])) * total:
                token = x
                break
        accepted.append(t - r0)
        nxt.append(token if token >= 0 else last)
    return accepted, nxt
