"""The pool's and the verification's entry points without a GPU: bad arguments are refused with
the documented status before any device call, empty problems are no-ops, and the workspace sizes
follow their formulas."""
import ctypes

import pytest
import torch

from exact_io_aware_13_gb300 import _lib
from exact_io_aware_13_gb300 import build as libbuild

OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 5
NAMES = ("k", "v", "exp", "k2", "v2", "exp2", "table", "lens", "refs", "new", "out", "map", "ws", "p", "q",
         "tok", "offs", "u", "su", "acc", "next", "kept")
PTR = {n: 0x10000000 * (i + 1) for i, n in enumerate(NAMES)}


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def _cache(kind=0, d=64, ps=16, pages=10, Hkv=2, maxp=8, two="", **kw):
    p = dict({n: PTR[n + two] for n in ("k", "v")}, exp=PTR["exp" + two] if kind == 1 else None)
    p.update(kw)
    return _lib.PagedCache(p["k"], p["v"], p["exp"], None, kind, pages, Hkv, ps, d, maxp)


def _fork(lib, B=3, maxp=8, pages=10, ps=16, wsb=1 << 30, **kw):
    p = {**PTR, **kw}
    return lib.attn_cache_fork(p["table"], p["lens"], p["refs"], p["new"], B, maxp, pages, ps, p["ws"],
                               wsb, None)


def _resize(lib, cache, B=3, window=0, wsb=1 << 30, **kw):
    p = {**PTR, **kw}
    return lib.attn_cache_resize(cache and ctypes.byref(cache), p["table"], p["lens"], p["refs"], p["new"],
                                 B, window, p["out"], p["ws"], wsb, None)


def _compact(lib, cache, B=3, wsb=1 << 30, **kw):
    p = {**PTR, **kw}
    return lib.attn_cache_compact(cache and ctypes.byref(cache), p["table"], p["lens"], p["refs"], B,
                                  p["out"], p["map"], p["ws"], wsb, None)


def _copy(lib, a, b, n=3, wsb=1 << 30, **kw):
    p = {**PTR, **kw}
    return lib.attn_cache_copy(a and ctypes.byref(a), b and ctypes.byref(b), p["new"], p["out"], n,
                               p["ws"], wsb, None)


def _verify(lib, kind=0, B=2, T=5, V=100, ps=100, qs=100, **kw):
    p = {**PTR, **kw}
    return lib.attn_verify_drafts(kind, p["p"], ps, p["q"], qs, p["tok"], p["offs"], p["u"], p["su"],
                                  p["lens"], B, T, V, p["acc"], p["next"], p["kept"], None)


@pytest.mark.parametrize("call", [_resize, _compact])
def test_bad_caches(lib, call):
    assert call(lib, None) == ARG
    assert call(lib, _cache(kind=2)) == ARG
    assert call(lib, _cache(1, exp=None)) == ARG
    assert call(lib, _cache(0, exp=PTR["exp"])) == ARG
    assert call(lib, _cache(d=96)) == SHAPE
    for ps in (0, 4, 12, 48, -16):
        assert call(lib, _cache(ps=ps)) == SHAPE, ps
    for bad in (dict(pages=-1), dict(Hkv=-1), dict(maxp=-1), dict(pages=1 << 30)):
        assert call(lib, _cache(**bad)) == SHAPE, bad
    assert call(lib, _cache(), B=-1) == SHAPE
    for name in ("k", "v"):
        assert call(lib, _cache(**{name: None})) == ARG
        assert call(lib, _cache(**{name: PTR[name] + 8})) == ALIGN
    assert call(lib, _cache(1, exp=PTR["exp"] + 8)) == ALIGN
    for name in ("table", "lens", "refs", "out"):
        assert call(lib, _cache(), **{name: None}) == ARG, name
        assert call(lib, _cache(), **{name: PTR[name] + 2}) == ALIGN, name
    assert call(lib, _cache(), ws=None) == WORKSPACE
    assert call(lib, _cache(), ws=PTR["ws"] + 128) == ALIGN


def test_resize_refusals(lib):
    assert _resize(lib, _cache(), window=-1) == ARG
    assert _resize(lib, _cache(), new=None) == ARG
    assert _resize(lib, _cache(), new=PTR["new"] + 1) == ALIGN
    need = lib.attn_resize_workspace_size(3, 8, 10)
    assert _resize(lib, _cache(), wsb=need - 1) == WORKSPACE


def test_compact_refusals(lib):
    assert _compact(lib, _cache(), map=None) == ARG
    assert _compact(lib, _cache(), wsb=lib.attn_compact_workspace_size(10) - 1) == WORKSPACE


def test_fork_refusals(lib):
    for bad in (dict(B=-1), dict(B=49153), dict(maxp=-1), dict(pages=-1), dict(ps=0), dict(ps=12)):
        assert _fork(lib, **bad) == SHAPE, bad
    for name in ("table", "lens", "refs", "new"):
        assert _fork(lib, **{name: None}) == ARG, name
        assert _fork(lib, **{name: PTR[name] + 2}) == ALIGN, name
    assert _fork(lib, wsb=lib.attn_fork_workspace_size(3, 8) - 1) == WORKSPACE
    assert _fork(lib, ws=None) == WORKSPACE
    assert _fork(lib, ws=PTR["ws"] + 16) == ALIGN
    assert _fork(lib, B=0, table=None, lens=None, new=None, ws=None) == OK


def test_copy_refusals(lib):
    a, b = _cache(), _cache(two="2")
    assert _copy(lib, None, b) == ARG and _copy(lib, a, None) == ARG
    assert _copy(lib, a, _cache(1, two="2")) == ARG
    for bad in (dict(d=128), dict(Hkv=1), dict(ps=32)):
        assert _copy(lib, a, _cache(two="2", **bad)) == SHAPE
    assert _copy(lib, a, b, n=-1) == SHAPE
    assert _copy(lib, a, b, n=0, new=None, out=None, ws=None) == OK
    assert _copy(lib, a, b, new=None) == ARG and _copy(lib, a, b, out=None) == ARG
    assert _copy(lib, a, b, new=PTR["new"] + 2) == ALIGN
    assert _copy(lib, a, b, wsb=lib.attn_copy_workspace_size(10, 3) - 1) == WORKSPACE
    size = 10 * 2 * 16 * 64 * 2                               # bytes of K
    for k in (PTR["k"] + size - 16, PTR["k"] + 4096, PTR["k"] - size + 16, PTR["v"] + 16):
        assert _copy(lib, a, _cache(two="2", k=k)) == ARG     # pools that overlap
    assert _copy(lib, a, _cache(k=PTR["k"], v=PTR["v2"])) == ARG


def test_verify_refusals(lib):
    assert _verify(lib, kind=3) == ARG
    for bad in (dict(B=-1), dict(T=-1), dict(V=-1), dict(ps=-1), dict(qs=-100), dict(B=(1 << 26) + 1)):
        assert _verify(lib, **bad) == SHAPE, bad
    for name in ("p", "tok", "offs", "u", "su", "acc", "next"):
        assert _verify(lib, **{name: None}) == ARG, name
    assert _verify(lib, lens=None) == ARG                     # seq_lens and kept_lens go together
    assert _verify(lib, kept=None) == ARG
    assert _verify(lib, p=PTR["p"] + 2) == ALIGN
    assert _verify(lib, kind=1, q=PTR["q"] + 1) == ALIGN
    for name in ("tok", "offs", "u", "su", "acc", "next", "kept", "lens"):
        assert _verify(lib, **{name: PTR[name] + 2}) == ALIGN, name
    assert _verify(lib, B=0, offs=None, su=None, acc=None, next=None) == OK


def test_workspace_sizes(lib):
    r = lambda n: -(-n // 256) * 256  # noqa: E731
    for B, M, pages, n in ((0, 0, 0, 0), (1, 1, 1, 1), (100, 33, 5000, 777), (7, 1000, 123_457, 64)):
        assert lib.attn_fork_workspace_size(B, M) == (r(4 * B * M) + 2 * r(4 * B) if B else 0)
        assert lib.attn_resize_workspace_size(B, M, pages) == (
            6 * r(4 * B) + 2 * r(4 * pages) + r(4 * min(pages, B * M)) + 256)
        assert lib.attn_compact_workspace_size(pages) == 2 * r(4 * pages) + 256
        assert lib.attn_copy_workspace_size(pages, n) == r(4 * pages)
    assert lib.attn_fork_workspace_size(-1, 5) == 0
    assert lib.attn_resize_workspace_size(1, -1, 5) == 0
    assert lib.attn_compact_workspace_size(-1) == lib.attn_copy_workspace_size(1, -1) == 0


def test_the_binding_refuses_wrong_tensors():
    import exact_io_aware_13_gb300 as ea
    z = torch.zeros
    i = lambda *s: z(s, dtype=torch.int32)  # noqa: E731
    kv = z(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ea.cache_fork(i(2, 3), i(2), i(4), i(2), page_size=16)
    with pytest.raises(ValueError, match="page_table must be torch.int32"):
        ea.cache_fork(z(2, 3), i(2), i(4), i(2), page_size=16)
    with pytest.raises(ValueError, match="k_cache must be torch.uint8"):
        ea.cache_resize(kv, kv, i(2, 3), i(2), i(4), i(2), kv_exp=z(4, 2, 16, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="must be a tensor"):
        ea.cache_compact(None, kv, i(2, 3), i(2), i(4))
    with pytest.raises(ValueError, match="target must be"):
        ea.verify_drafts(z(3, 10, dtype=torch.float64), i(3), i(2), z(3), z(1))
    with pytest.raises(ValueError, match="missing"):
        ea.cache_resize_into(kv, kv, i(2, 3), i(2), i(4), i(2), None, None)
    with pytest.raises(ValueError, match="used and page_map"):
        ea.cache_compact_into(kv, kv, i(2, 3), i(2), i(4), None, None, None)
    with pytest.raises(ValueError, match="accepted"):
        ea.verify_drafts_into(z(3, 10), i(3), i(2), z(3), z(1), None, None)

