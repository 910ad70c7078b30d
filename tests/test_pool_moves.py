"""Move lists of plans that many CTAs share, and the copies of pages that are small and many: every
byte of the caches, those behind a partial page's copied tokens too."""
import numpy as np
import pytest
import torch

from tests.pool_inputs import PoolPair

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# Runs below 4 KB per tensor are copied a piece per lane when a call's bound on its 8 KB pieces
# exceeds 64 per SM: a resize counts K, V and the scales of each row and head, a compaction those
# of half of the pool's pages.
PER_SM = 64


@pytest.mark.parametrize("kind,page,d", [("e4m3", 16, 128),   # 2048 bytes of codes and 32 of scales
                                         ("e4m3", 8, 64), ("e4m3", 32, 64), ("bf16", 8, 128),
                                         ("bf16", 16, 64)])
def test_many_partial_pages(kind, page, d):
    """Forked rows of odd lengths all write at once: the copies of their partial pages."""
    ea = _ea()
    per_row = 3 if kind == "e4m3" else 2
    Hkv, group = 5, 3
    B = -(-(PER_SM * sms() + 1) // (per_row * Hkv * group)) * group
    w = PoolPair(B, 4, B * 3 + 50, Hkv=Hkv, page=page, d=d, kind=kind, seed=page + d)
    lens = [0] * B
    for b in range(0, B, group):                              # every partial length, a full page too
        lens[b] = int(w.rng.integers(0, 2)) * page + 1 + b // group % page
    assert w.resize(ea, lens)[0] == 0
    w.fork(ea, [b // group * group for b in range(B)])
    missing, copies = w.resize(ea, [L + 1 for L in w.lens])
    assert missing == 0 and len(copies) > B // 2
    assert len({c[2] for c in copies}) == page - 1
    w.check()
    w.holders()
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind,page,d,Hkv", [("e4m3", 16, 64, 1), ("bf16", 8, 64, 1), ("bf16", 8, 128, 1),
                                             ("e4m3", 8, 64, 3)])
def test_many_small_pages_are_compacted(kind, page, d, Hkv):
    ea = _ea()
    per_page = 3 if kind == "e4m3" else 2
    pages = 2 * (-(-(PER_SM * sms() + 1) // per_page)) + 3
    B, M = 60, 100
    w = PoolPair(B, M, pages, Hkv=Hkv, page=page, d=d, kind=kind, seed=pages)
    # rows in random places of the pool, pages that no row holds too
    perm = w.rng.permutation(pages)
    for b in range(B):
        w.lens[b] = int(w.rng.integers(0, M * page + 1))
        n = -(-w.lens[b] // page)
        w.table[b][:n], perm = perm[:n].tolist(), perm[n:]
        for p in w.table[b][:n]:
            w.refs[p] += 1
    for p in perm[:len(perm) // 4].tolist():
        w.refs[p] = 2
    w.to_gpu()
    _, moves = w.compact(ea)
    assert len(moves) > 1000
    w.check()
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,M,pages", [(700, 30, 26_000), (90, 200, 40_000)])
def test_plans_of_many_ctas(kind, B, M, pages):
    """A run of the operators over more pages than one CTA plans, with partial pages to copy."""
    ea = _ea()
    w = PoolPair(B, M, pages - 1, page=8, d=64, Hkv=1, kind=kind, seed=B, window=60)
    most, copied, moved = min(M * 8, (pages * 8) // B), 0, 0
    for step in range(3):
        copied += len(w.resize(ea, w.random_lens(most))[1])
        w.check(f"{step}: resize")
        w.fork(ea, w.random_parents())
        missing, copies = w.resize(ea, [min(L + 1, M * 8) for L in w.lens])
        copied += len(copies)
        w.check(f"{step}: fork, resize")
        moved += len(w.compact(ea)[1])
        w.check(f"{step}: compact")
        w.holders()
    assert copied > B // 4 and moved > 100
    assert ea.device_status() == 0
