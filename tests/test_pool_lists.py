"""A caller's list of page copies: the rules about repeated destinations, sources that are
destinations, copies of a page to itself and pages outside of the pools are the same for lists of
every length, what is copied as well as what is reported."""
import numpy as np
import pytest
import torch

from oracle import pool_oracle as P
from tests.pool_inputs import PoolPair

pytestmark = pytest.mark.gpu

BAD_INPUT = 8
PADDED = [0, 33, 64, 1024, 1025, 4000]                        # entries; 0: the list as it is


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rules(src, dst, pages_from, pages_to, same):
    """(copies, whether an entry is reported), from the statement of attn_cache_copy."""
    entries = [(i, s, d) for i, (s, d) in enumerate(zip(src, dst)) if s >= 0 and d >= 0]
    inside = [(i, s, d) for i, s, d in entries if s < pages_from and d < pages_to]
    bad = any(s >= pages_from or d >= pages_to for s, d in zip(src, dst))
    copies = []
    for i, s, d in inside:
        first = all(j >= i or e != d for j, _, e in inside)
        read = same and s != d and any(j != i and e == s for j, _, e in inside)
        if first and not read:
            copies.append((s, d))
        else:
            bad = True
    return copies, bad


def check(src, dst, same, n, kind="e4m3", Hkv=1):
    """The list, spread over n entries with skipped ones between, through the call and the rules."""
    ea = _ea()
    if n:
        at = np.sort(np.random.default_rng(n).permutation(n)[:len(src)])
        s, d = np.full(n, -1), np.full(n, 3)
        s[at], d[at] = src, dst
        src, dst = s.tolist(), d.tolist()
    a = PoolPair(1, 1, 40, page=8, Hkv=Hkv, kind=kind, seed=1)
    b = a if same else PoolPair(1, 1, 50, page=8, Hkv=Hkv, kind=kind, seed=2)
    copies, bad = rules(src, dst, 40, 40 if same else 50, same and Hkv > 0)
    P.copy_pages(a.cache, b.cache, copies)
    ea.cache_copy(*a.g_cache[:2], *b.g_cache[:2], i32(src), i32(dst), kv_exp=a.g_cache[2],
                  kv_exp_to=b.g_cache[2])
    assert ea.device_status() == (BAD_INPUT if bad else 0)
    a.check()
    b.check()


LISTS = {
    "plain": ([1, 2, 3], [20, 21, 22]),
    "repeated": ([1, 2, 3, 2], [20, 21, 20, 21]),
    "repeated alike": ([1, 2, 1], [20, 21, 20]),
    "outside": ([1, 40, 2, 3], [20, 21, 50, 22]),
    "chain": ([5, 20, 6], [20, 22, 30]),
    "swap": ([5, 6], [6, 5]),
    "to itself": ([7, 2], [7, 20]),
    "to itself twice": ([7, 2, 7], [7, 20, 7]),
    "over, then itself": ([1, 7, 2], [7, 7, 20]),
    "itself, then over": ([7, 1, 2], [7, 7, 20]),
    "from one that stays": ([7, 7], [7, 20]),
}


@pytest.mark.parametrize("n", PADDED)
@pytest.mark.parametrize("same", [True, False])
@pytest.mark.parametrize("name", list(LISTS))
def test_rules(name, same, n):
    check(*LISTS[name], same, n)


@pytest.mark.parametrize("n", PADDED)
@pytest.mark.parametrize("same", [True, False])
def test_rules_of_pages_without_bytes(same, n):
    """Pools without heads count as two: there is nothing to copy, and the entries left out are reported."""
    for name in ("plain", "repeated", "to itself twice", "chain"):
        check(*LISTS[name], same, n, Hkv=0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("same", [True, False])
@pytest.mark.parametrize("entries", [12, 32, 33, 300, 1024, 1025, 2500])
def test_random_lists(entries, same, kind):
    """Entries at random: most destinations repeat, some pages lie outside."""
    rng = np.random.default_rng(entries)
    for _ in range(3):
        check(rng.integers(-3, 41, entries).tolist(), rng.integers(-3, 51, entries).tolist(), same, 0, kind,
              Hkv=2)


@pytest.mark.parametrize("n", PADDED)
@pytest.mark.parametrize("pages_from,pages_to", [(40, 25), (25, 40)])
def test_one_pool_in_two_sizes(pages_from, pages_to, n):
    """A pool beside its own front: every page that the one or the other has can be copied."""
    ea = _ea()
    for src, dst in (([39, 1, 30, 24], [5, 2, 24, 6]), ([3, 1, 24], [39, 30, 20]), ([39, 5], [25, 39]),
                     ([30, 2], [3, 30])):
        if n:
            at = np.sort(np.random.default_rng(n).permutation(n)[:len(src)])
            s, d = np.full(n, -1), np.full(n, 3)
            s[at], d[at] = src, dst
            src, dst = s.tolist(), d.tolist()
        a = PoolPair(1, 1, 40, page=8, Hkv=1, kind="e4m3", seed=1)
        copies, bad = rules(src, dst, pages_from, pages_to, True)
        P.copy_pages(a.cache, a.cache, copies)
        k, v, exp = a.g_cache
        ea.cache_copy(k[:pages_from], v[:pages_from], k[:pages_to], v[:pages_to], i32(src), i32(dst),
                      kv_exp=exp[:pages_from], kv_exp_to=exp[:pages_to])
        assert ea.device_status() == (BAD_INPUT if bad else 0)
        a.check()
