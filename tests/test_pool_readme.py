"""The serving loop as README prints it: with room for the new tokens, and in a pool that is full,
where it may neither overwrite cached tokens nor lose any."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def printed(lines):
    """README's block with the pool's calls, the given number of its last lines left out."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = [b for b in blocks if "cache_fork" in b]
    return block.rstrip().rsplit("\n", lines)[0] if lines else block


def loop_state(kind, spare, seed=0):
    """Three beams of one prompt and two sequences of their own, over a pool with `spare` free pages."""
    import exact_io_aware_13_gb300 as ea
    g = torch.Generator("cuda").manual_seed(seed)
    B, M, Hkv, page, d, V = 5, 6, 2, 64, 64, 200
    lens = [150, 0, 0, 64, 200]
    pages = sum(-(-n // page) for n in lens) + spare
    e4m3 = kind == "e4m3"
    def pool():
        shape = (pages, Hkv, page, d)
        if e4m3:
            return torch.zeros(shape, dtype=torch.uint8, device="cuda")
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    exps = [torch.zeros(pages, Hkv, page, 2, dtype=torch.uint8, device="cuda") if e4m3 else None for _ in "ab"]
    n_new = i32([4, 1, 3, 2, 5])
    offsets = torch.cat([i32([0]), n_new.cumsum(0).int()])
    T = int(offsets[-1])
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    st = dict(
        ea=ea, k_cache=pool(), v_cache=pool(), k_to=pool(), v_to=pool(), kv_exp=exps[0], kv_exp_to=exps[1],
        table=torch.full((B, M), -1, dtype=torch.int32, device="cuda"), lens=i32([0] * B),
        refs=torch.zeros(pages, dtype=torch.int32, device="cuda"), parents=i32([0, 0, 0, 3, 4]),
        n_new=n_new, offsets=offsets, k=(rand(T, Hkv, d) - 0.5).bfloat16(), v=(rand(T, Hkv, d) - 0.5).bfloat16(),
        probs=torch.softmax(2 * rand(T, V), -1), draft_probs=torch.softmax(2 * rand(T, V), -1),
        tokens=torch.randint(0, V, (T,), generator=g, device="cuda").int(), u_accept=rand(T), u_sample=rand(B),
        src_pages=i32([0]), dst_pages=i32([0]))
    c = (st["k_cache"], st["v_cache"])
    assert ea.cache_resize(*c, st["table"], st["lens"], st["refs"], i32(lens), kv_exp=st["kv_exp"]).tolist() == [0]
    x = (rand(sum(lens), Hkv, d) - 0.5).bfloat16()
    ea.cache_write(x, -x, *c, st["table"], torch.cat([i32([0]), i32(lens).cumsum(0).int()]), st["lens"],
                   kv_exp=st["kv_exp"])
    return st


def read_back(st):
    lens = st["lens"]
    offs = torch.cat([i32([0]), lens.cumsum(0).int()])
    return st["ea"].cache_read(st["k_cache"], st["v_cache"], st["table"], offs, lens, int(offs[-1]),
                               kv_exp=st["kv_exp"])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_with_room(kind):
    st = loop_state(kind, spare=20)
    exec(printed(0), st)
    assert st["lacking"].tolist() == [0]
    new = st["n_new"].tolist()
    assert st["lens"].tolist() == [L + 1 + a for L, a in zip([150, 150, 150, 64, 200], st["accepted"].tolist())]
    assert all(0 <= a < n for a, n in zip(st["accepted"].tolist(), new)) and min(st["token"].tolist()) >= 0
    assert st["ea"].device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_in_a_full_pool(kind):
    """Beams share a partly filled page and a sequence needs a new one, and none is free."""
    st = loop_state(kind, spare=0)
    ea, page_table = st["ea"], st["table"]
    ea.cache_fork(page_table, st["lens"], st["refs"], st["parents"], page_size=64)
    st["parents"] = i32(range(5))
    before = [x.clone() for x in (*read_back(st), st["lens"], st["refs"], page_table)]
    exec(printed(2), st)                                      # (without the compaction and the copy)
    assert st["lacking"].item() > 0
    after = (*read_back(st), st["lens"], st["refs"], page_table)
    for x, y in zip(before, after):
        assert torch.equal(x, y)
    assert st["accepted"].tolist() == [0] * 5 and st["token"].tolist() == [-1] * 5
    # scoring the batch that has lost its rows writes none, in one chunk of keys or in several
    T, cap = st["k"].shape[0], 6 * 64
    for split in (cap, 128):
        o = torch.full((T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, 4), 7.0, device="cuda")
        ws = torch.empty(ea.prefill_workspace_size(T, 4, 64, cap, split), dtype=torch.uint8, device="cuda")
        ea.prefill_paged_into(torch.ones_like(o), st["k_cache"], st["v_cache"], page_table, st["rows"], st["lens"], o,
                              lse, ws, max_new=T, max_seq_len=cap, split_keys=split, scale=0.125,
                              kv_exp=st["kv_exp"], mask_kind=ea.MASK_CAUSAL)
        assert bool((o == 7).all()) and bool((lse == 7).all())
    assert ea.device_status() == 0
