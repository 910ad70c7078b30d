"""GPU parity of the pool's operators (fork, resize, compact, copy) against plain loops: every
integer and every byte of the caches has to be the same."""
import numpy as np
import pytest
import torch

from oracle import pool_oracle as P
from tests.pool_inputs import PoolPair

pytestmark = pytest.mark.gpu

BAD_INPUT = 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,M,pages,page,d,Hkv,window", [
    (1, 1, 1, 8, 64, 1, 0), (1, 7, 9, 16, 128, 3, 0), (5, 6, 40, 8, 64, 2, 0),
    (9, 12, 60, 32, 64, 1, 70), (33, 20, 300, 8, 64, 1, 0), (40, 9, 200, 16, 64, 2, 1),
    (7, 3, 24, 192, 64, 2, 0), (64, 40, 1500, 8, 64, 1, 100), (3, 70, 250, 64, 128, 1, 0)])
def test_walk(kind, B, M, pages, page, d, Hkv, window):
    """A random run of the operators as a serving loop makes them."""
    ea = _ea()
    w = PoolPair(B, M, pages, page=page, d=d, Hkv=Hkv, kind=kind, seed=B + M + pages, window=window)
    refused = 0
    for step in range(14):
        what = f"step {step}"
        op = ("resize", "fork", "resize", "compact")[step % 4]
        if op == "resize":
            refused += w.resize(ea, w.random_lens())[0] > 0
        elif op == "fork":
            w.fork(ea, w.random_parents())
        else:
            w.compact(ea)
        w.check(f"{what}: {op}")
        w.holders()
    assert ea.device_status() == 0


@pytest.mark.parametrize("B,M,pages,page", [(1000, 24, 9000, 8), (300, 400, 150_000, 16),
                                            (5, 30_000, 130_000, 8), (3000, 3, 5000, 32)])
def test_large_states(B, M, pages, page):
    """Several CTAs share the work; rows and pages are no multiples of theirs."""
    ea = _ea()
    w = PoolPair(B, M, pages - 1, page=page, Hkv=0, seed=B)
    most = min(M * page, (pages * page) // B)
    for step in range(3):
        w.resize(ea, w.random_lens(most))
        w.check()
        w.fork(ea, w.random_parents())
        w.check()
        w.compact(ea)
        w.check()
    assert ea.device_status() == 0


def test_copy_on_write_rules():
    """Rows 0-2 share a last page that is partly filled, rows 3-4 another one that a kept prefix
    holds too, row 5 holds its own."""
    ea = _ea()
    w = PoolPair(6, 4, 30, page=16, seed=3)
    w.resize(ea, [20, 0, 0, 33, 0, 5])
    w.fork(ea, [0, 0, 0, 3, 3, 5])
    kept = w.table[3][2]
    w.refs[kept] += 1
    w.g_refs[kept] += 1
    shared = w.table[0][1]
    _, copies = w.resize(ea, [21, 21, 20, 34, 34, 6])         # row 2 keeps the page it reads
    w.check()
    assert [c[0] for c in copies] == [shared, shared, kept, kept]
    _, copies = w.resize(ea, [21, 21, 21, 34, 34, 6])         # row 2 is its only holder now
    w.check()
    assert copies == [] and w.table[2][1] == shared
    w.holders(extra=1)
    # two holders, both write: the lower row keeps the page
    w.resize(ea, [21, 21, 0, 34, 34, 6])
    w.fork(ea, [0, 0, 1, 3, 4, 5])
    pages = [r[1] for r in w.table[:3]]
    assert pages[0] == pages[1]
    _, copies = w.resize(ea, [40, 22, 22, 34, 34, 6])
    w.check()
    assert [c[0] for c in copies] == [pages[0]] and w.table[0][1] == pages[0]
    assert ea.device_status() == 0


def test_a_rollback_lets_its_neighbour_keep_the_page():
    ea = _ea()
    w = PoolPair(2, 4, 10, page=8, seed=4)
    w.resize(ea, [12, 0])
    w.fork(ea, [0, 0])
    _, copies = w.resize(ea, [13, 8])                         # row 1 drops the shared page
    w.check()
    assert copies == []


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_shortage_changes_nothing(kind):
    ea = _ea()
    w = PoolPair(4, 8, 10, page=16, kind=kind, seed=5, window=20)
    assert w.resize(ea, [60, 30, 0, 0])[0] == 0
    w.fork(ea, [0, 1, 1, -1])
    before = [x.clone() for x in w.state]
    # rows 1 and 2 write into a shared page: 1 copy; row 3 asks for 8 pages; row 0 gives back
    missing, _ = w.resize(ea, [17, 31, 31, 128])
    assert missing > 0
    w.check()
    assert all(torch.equal(a, b) for a, b in zip(before, w.state))
    assert w.resize(ea, [17, 31, 31, 128 - 16 * missing])[0] == 0  # the last page is handed out
    w.check()
    assert 0 not in w.refs
    assert ea.device_status() == 0


def test_a_window_gives_pages_back():
    """Pages that the window has passed are free, once; a fork takes the row as it is."""
    ea = _ea()
    w = PoolPair(3, 40, 60, page=8, seed=6)
    w.resize(ea, [100, 0, 300], window=0)
    for n in range(1, 12):
        w.resize(ea, [100 + 5 * n, 0, max(0, 300 - 31 * n)], window=50)
        w.check()
        w.holders()
    w.fork(ea, [0, 0, 0])
    w.check()
    w.resize(ea, [200, 157, 156], window=50)
    w.check()
    w.holders()
    assert any(e < 0 for e in w.table[0][:20])
    w.resize(ea, [0, 0, 0], window=50)
    w.check()
    assert sum(w.refs) == 0
    assert ea.device_status() == 0


def test_fork_permutes_and_frees():
    ea = _ea()
    w = PoolPair(6, 5, 40, page=8, seed=7)
    w.resize(ea, [0, 40, 17, 8, 1, 33])
    w.fork(ea, [5, 0, 1, 2, 3, 4])
    w.check()
    w.fork(ea, [3, 3, -1, 3, -7, 5])
    w.check()
    w.holders()
    w.fork(ea, [-1] * 6)
    w.check()
    assert sum(w.refs) == 0
    assert ea.device_status() == 0


def test_most_rows():
    """As many rows as a fork takes, against array operations."""
    ea, B, page = _ea(), 49152, 8
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 3, B) * page                       # whole pages: nothing is copied
    k = torch.zeros(B * 2 + 50, 1, page, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    g_lens, refs = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(len(k), dtype=torch.int32,
                                                                                device="cuda")
    assert ea.cache_resize(k, k.clone(), table, g_lens, refs, i32(lens)).tolist() == [0]
    want = np.full((B, 4), -1)
    need, at = lens // page, np.concatenate([[0], np.cumsum(lens // page)])
    for i in (0, 1):
        want[need > i, i] = at[:-1][need > i] + i
    assert np.array_equal(table.cpu().numpy(), want) and np.array_equal(g_lens.cpu().numpy(), lens)
    assert int(refs.sum()) == int(need.sum()) == int(refs[:at[-1]].sum())
    parents = rng.integers(-1, B, B)
    ea.cache_fork(table, g_lens, refs, i32(parents), page_size=page)
    took = np.where(parents[:, None] >= 0, want[parents], -1)
    assert np.array_equal(table.cpu().numpy(), took)
    assert np.array_equal(g_lens.cpu().numpy(), np.where(parents >= 0, lens[parents], 0))
    assert np.array_equal(refs.cpu().numpy(), np.bincount(took[took >= 0], minlength=len(k)))
    used, page_map = ea.cache_compact(k, k.clone(), table, g_lens, refs)
    held = np.unique(took[took >= 0])
    assert used.tolist() == [len(held)]
    m = page_map.cpu().numpy()
    assert np.array_equal(table.cpu().numpy(), np.where(took >= 0, m[took], -1))
    assert np.array_equal(np.sort(m[held]), np.arange(len(held))) and int((m >= 0).sum()) == len(held)
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_holders_outside_of_the_table(kind):
    """A kept page that no row holds moves too, with its count, and is never handed out."""
    ea = _ea()
    w = PoolPair(2, 6, 20, page=8, kind=kind, seed=12)
    w.resize(ea, [16, 40])
    for p, n in ((17, 3), (19, 1), (3, 2)):
        w.refs[p] += n
        w.g_refs[p] += n
    w.resize(ea, [48, 48])
    w.check()
    w.resize(ea, [0, 9])
    used, moves = w.compact(ea)
    w.check()
    assert used == 4 and {m[0] for m in moves} == {17, 19}      # 2 and 3 (kept too), 17, 19
    w.holders(extra=6)
    assert ea.device_status() == 0


def test_lengths_at_the_ends_of_their_type():
    ea = _ea()
    big, small = 2 ** 31 - 1, -2 ** 31
    for lens, new in (([big, 3], [0, 3]), ([small, 3], [0, 3]), ([5, 3], [big, 3]), ([5, 3], [small, 3])):
        w = PoolPair(2, 4, 12, page=8, seed=13)
        w.resize(ea, [5, 3])
        w.g_lens.copy_(i32(lens))
        ea.cache_resize(*w.g_cache[:2], *w.state, i32(new), window=big)
        assert ea.device_status() == BAD_INPUT
        assert int(w.g_lens[1]) == 3
    w = PoolPair(2, 4, 12, page=8, seed=13)
    w.resize(ea, [5, 3])
    w.fork(ea, [small, 0])
    w.check()
    w.resize(ea, [0, 32], window=big)
    w.check()
    assert ea.device_status() == 0


def test_the_binding_refuses():
    ea = _ea()
    w, e = PoolPair(2, 3, 6, page=8), PoolPair(2, 3, 6, page=8, kind="e4m3")
    k, v = w.g_cache[:2]
    one = i32([0])
    for bad in (dict(page_table=w.g_table[:, :2]), dict(page_table=w.g_table.long()), dict(seq_lens=i32([0])),
                dict(page_refs=i32([0] * 5)), dict(new_lens=i32([1])), dict(new_lens=w.g_lens.cpu()),
                dict(k_cache=k[:, :, :4]), dict(v_cache=v[:5]), dict(kv_exp=e.g_cache[2])):
        args = dict(k_cache=k, v_cache=v, page_table=w.g_table, seq_lens=w.g_lens, page_refs=w.g_refs,
                    new_lens=i32([1, 1]))
        args.update(bad)
        with pytest.raises(ValueError):
            ea.cache_resize(**args)
    for bad in (dict(kv_exp_to=e.g_cache[2]), dict(kv_exp=e.g_cache[2]), dict(src_pages=i32([0, 1])),
                dict(dst_pages=one.float()), dict(k_to=PoolPair(1, 1, 6, page=16).g_cache[0])):
        args = dict(k_cache=k, v_cache=v, k_to=k, v_to=v, src_pages=one, dst_pages=one)
        args.update(bad)
        with pytest.raises(ValueError):
            ea.cache_copy(**args)
    with pytest.raises(ValueError, match="both be given"):
        ea.cache_copy(*e.g_cache[:2], k, v, one, one, kv_exp=e.g_cache[2])
    with pytest.raises(ea.AttnError):                         # a part of the pool itself
        ea.cache_copy(k, v, k[1:], v[1:], one, one)
    with pytest.raises(ea.AttnError):
        ea.cache_resize(k, v, *w.state, i32([1, 1]), window=-1)
    with pytest.raises(ea.AttnError):
        ea.cache_fork(*w.state, i32([0, 1]), page_size=12)
    with pytest.raises(ea.AttnError):
        ea.cache_fork(*w.state, i32([0, 1]), page_size=8, workspace=torch.empty(8, device="cuda"))
    w.check()


# ------------------------------------------------------------------ copy
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,d,Hkv", [(8, 64, 1), (16, 128, 3), (64, 128, 8), (192, 64, 5)])
def test_copy_between_pools(kind, page, d, Hkv):
    ea = _ea()
    a = PoolPair(1, 1, 23, page=page, d=d, Hkv=Hkv, kind=kind, seed=1)
    b = PoolPair(1, 1, 31, page=page, d=d, Hkv=Hkv, kind=kind, seed=2)
    src, dst = [0, 22, 7, -1, 3, 7, 9], [30, 0, 7, 4, -2, 8, 22]
    moves = [(s, t) for s, t in zip(src, dst) if s >= 0 and t >= 0]
    P.copy_pages(a.cache, b.cache, moves)
    ea.cache_copy(*a.g_cache[:2], *b.g_cache[:2], i32(src), i32(dst), kv_exp=a.g_cache[2],
                  kv_exp_to=b.g_cache[2])
    assert ea.device_status() == 0
    a.check()
    b.check()


def test_copy_within_a_pool():
    ea = _ea()
    w = PoolPair(1, 1, 40, page=16, seed=9)
    src, dst = [1, 2, 3, 9], [20, 0, 21, 9]                   # (9 to itself: nothing to do)
    P.copy_pages(w.cache, w.cache, [(1, 20), (2, 0), (3, 21)])
    ea.cache_copy(*w.g_cache[:2], *w.g_cache[:2], i32(src), i32(dst))
    assert ea.device_status() == 0
    w.check()
    # 20 is the destination of 1 and the source of 22; 30 has two sources, the first counts
    P.copy_pages(w.cache, w.cache, [(5, 20), (6, 30)])
    ea.cache_copy(*w.g_cache[:2], *w.g_cache[:2], i32([5, 20, 6, 7, 40]), i32([20, 22, 30, 30, 1]))
    assert ea.device_status() == BAD_INPUT
    w.check()


def test_copy_many_pages():
    """More entries than threads, repeated destinations among them."""
    ea = _ea()
    a, b = (PoolPair(1, 1, 5000, page=8, Hkv=1, kind="e4m3", seed=s) for s in (1, 2))
    src = np.random.default_rng(3).integers(0, 5000, 9000)
    dst = np.random.default_rng(4).integers(0, 5000, 9000)
    first = {}
    for s, t in zip(src, dst):
        first.setdefault(int(t), int(s))
    P.copy_pages(a.cache, b.cache, [(s, t) for t, s in first.items()])
    ea.cache_copy(*a.g_cache[:2], *b.g_cache[:2], i32(src), i32(dst), kv_exp=a.g_cache[2],
                  kv_exp_to=b.g_cache[2])
    assert ea.device_status() == BAD_INPUT                    # the repeated ones are reported
    b.check()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes per tensor: pages at its far end move and are copied."""
    ea = _ea()
    pages, shape = 33_000, (8, 64, 128)                       # 128 KB a page: 4.3 GB
    k = torch.zeros((pages,) + shape, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for p in (0, 5, 32_766, 32_999):
        k[p], v[p] = p / 64, -p / 64 - 1
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[[5, 32_766, 32_999]] = i32([1, 2, 1])
    table, lens = i32([[32_999, 5, 32_766], [32_766, -1, -1]]), i32([192, 40])
    ea.cache_copy(k, v, k, v, i32([32_999, 5]), i32([32_998, 32_997]))
    assert ea.device_status() == 0
    assert bool((k[32_998] == k[32_999]).all()) and bool((v[32_997] == v[5]).all())
    used, page_map = ea.cache_compact(k, v, table, lens, refs)
    assert used.tolist() == [3] and refs[:3].tolist() == [1, 2, 1]
    assert table[0].tolist() == [0, 2, 1] and table[1].tolist() == [1, -1, -1]
    for p, old in ((0, 32_999), (1, 32_766), (2, 5)):
        assert int(page_map[old]) == p
        assert bool((k[p] == torch.tensor(old / 64).bfloat16().cuda()).all())
        assert bool((v[p] == torch.tensor(-old / 64 - 1).bfloat16().cuda()).all())
    # row 1 writes behind token 40 of page 1, which row 0 holds too: its copy goes to page 3
    missing = ea.cache_resize(k, v, table, lens, refs, i32([192, 41]))
    assert missing.tolist() == [0] and table[1, 0] == 3
    assert bool((k[3, :, :40] == k[1, :, :40]).all()) and bool((k[3, :, 40:] == 0).all())
    assert ea.device_status() == 0


# ------------------------------------------------------------------ bad inputs, empty ones
def test_bad_device_inputs_are_reported():
    ea = _ea()
    def fresh():
        w = PoolPair(3, 4, 12, page=8, seed=11)
        w.resize(ea, [20, 9, 0])
        assert ea.device_status() == 0
        return w
    w = fresh()
    ea.cache_fork(*w.state, i32([0, 7, 2]), page_size=8)      # no row 7: row 1 stays
    assert ea.device_status() == BAD_INPUT
    w.check()
    for lens in ([20, 9, 33], [20, -1, 0]):
        w = fresh()
        ea.cache_resize(*w.g_cache[:2], *w.state, i32(lens))
        assert ea.device_status() == BAD_INPUT
    for call in ("fork", "resize", "compact"):
        w = fresh()
        w.g_table[0, 1] = 12                                  # behind the pool
        if call == "fork":
            ea.cache_fork(*w.state, i32([1, 1, 0]), page_size=8)
        elif call == "resize":
            ea.cache_resize(*w.g_cache[:2], *w.state, i32([0, 10, 0]))
        else:
            ea.cache_compact(*w.g_cache[:2], *w.state)
        assert ea.device_status() == BAD_INPUT, call
        w = fresh()
        w.g_lens[1] = 33                                      # more than the table holds
        if call == "fork":
            ea.cache_fork(*w.state, i32([1, 0, 0]), page_size=8)
        elif call == "resize":
            ea.cache_resize(*w.g_cache[:2], *w.state, i32([21, 10, 0]))
        else:
            ea.cache_compact(*w.g_cache[:2], *w.state)
        assert ea.device_status() == BAD_INPUT, call
    w = fresh()
    w.g_table[0, 2] = -1                                      # no page where row 0 writes
    ea.cache_resize(*w.g_cache[:2], *w.state, i32([21, 9, 0]))
    assert ea.device_status() == BAD_INPUT


def test_empty_calls():
    ea = _ea()
    w = PoolPair(0, 3, 5, page=8)
    w.fork(ea, [])
    w.resize(ea, [])
    w.compact(ea)
    w.check()
    w = PoolPair(2, 0, 0, page=8)
    w.fork(ea, [1, 0])
    w.resize(ea, [0, 0])
    w.compact(ea)
    w.check()
    w = PoolPair(2, 3, 0, page=8)
    assert w.resize(ea, [9, 8])[0] == 3
    a = PoolPair(1, 1, 3, page=8)
    ea.cache_copy(*a.g_cache[:2], *a.g_cache[:2], i32([]), i32([]))
    a.check()
    assert ea.device_status() == 0
