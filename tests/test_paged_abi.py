"""The paged-cache entry points without a GPU: bad arguments are refused with the documented
status before any device call, empty problems are no-ops, and the sizes the library
computes follow their formulas."""
import ctypes

import pytest

from exact_io_aware_13_gb300 import _lib
from exact_io_aware_13_gb300 import build as libbuild

OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 5
PTR = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ("k", "v", "kc", "vc", "exp", "table", "offsets", "lens", "q", "o", "lse", "ws"))}


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def _cache(kind=0, d=64, ps=16, pages=10, Hkv=2, maxp=8, **kw):
    ptr = dict(PTR, exp=PTR["exp"] if kind == 1 else None)
    ptr.update(kw)
    return _lib.PagedCache(ptr["kc"], ptr["vc"], ptr["exp"], ptr["table"], kind, pages, Hkv, ps, d,
                           maxp)


def _write(lib, cache, T=5, B=2, kt=128, kh=64, vt=128, vh=64, **kw):
    p = {**PTR, **kw}
    return lib.attn_cache_write(cache and ctypes.byref(cache), p["k"], kt, kh, p["v"], vt, vh,
                                p["offsets"], p["lens"], B, T, None)


def _read(lib, cache, T=5, B=2, **kw):
    p = {**PTR, **kw}
    return lib.attn_cache_read(cache and ctypes.byref(cache), p["k"], p["v"], p["offsets"],
                               p["lens"], B, T, None)


def _prefill(lib, cache, T=5, B=2, Hq=4, new=5, msl=100, split=128, qt=256, qh=64, scale=0.1, mask=0,
             mp=None, score=0, sp=None, wsb=1 << 30, **kw):
    p = {**PTR, **kw}
    return lib.attn_prefill_paged(cache and ctypes.byref(cache), p["q"], qt, qh, p["o"], p["lse"],
                                  p["offsets"], p["lens"], B, T, Hq, new, msl, split,
                                  ctypes.c_float(scale), mask, mp, score, sp, p["ws"], wsb, None)


def _decode(lib, cache, B=2, Hq=4, Nq=1, msl=100, split=64, scale=0.1, mask=0, mp=None, score=0,
            sp=None, wsb=1 << 30, **kw):
    p = {**PTR, **kw}
    return lib.attn_decode_paged_e4m3(cache and ctypes.byref(cache), p["q"], p["lens"], p["o"],
                                      p["lse"], B, Hq, Nq, msl, split, ctypes.c_float(scale), mask,
                                      mp, score, sp, p["ws"], wsb, None)


CALLS = [_write, _read, _prefill]


@pytest.mark.parametrize("call", CALLS + [_decode])
def test_bad_caches(lib, call):
    kind = 1 if call is _decode else 0
    assert call(lib, None) == ARG
    assert call(lib, _cache(kind=2)) == ARG
    assert call(lib, _cache(kind, d=256)) == SHAPE
    assert call(lib, _cache(kind, d=96)) == SHAPE
    for ps in (0, 4, 12, 48, 96, -16):
        assert call(lib, _cache(kind, ps=ps, maxp=100)) == SHAPE, ps
    assert call(lib, _cache(kind, pages=-1)) == SHAPE
    assert call(lib, _cache(kind, Hkv=-2)) == SHAPE
    assert call(lib, _cache(kind, maxp=-1)) == SHAPE
    if call in (_prefill, _decode):                             # positions must fit 32 bits
        assert call(lib, _cache(kind, ps=64, maxp=1 << 25), msl=(1 << 31) - 1) == SHAPE
    assert call(lib, _cache(kind, pages=1 << 27)) == SHAPE      # over 2^31 cache rows
    assert call(lib, _cache(kind, pages=1 << 30, Hkv=8)) == SHAPE
    assert call(lib, _cache(1, exp=None)) == ARG                # codes without scales
    if call is not _decode:
        assert call(lib, _cache(0, exp=PTR["exp"])) == ARG      # scales of a bf16 cache
    for name in ("kc", "vc", "table"):
        assert call(lib, _cache(kind, **{name: None})) == ARG, name
    for name in ("kc", "vc"):
        assert call(lib, _cache(kind, **{name: 0x100008})) == ALIGN, name
    assert call(lib, _cache(kind, table=0x100002)) == ALIGN
    assert call(lib, _cache(1, exp=0x100008)) == ALIGN


@pytest.mark.parametrize("call", CALLS)
def test_bad_batches(lib, call):
    c = _cache()
    assert call(lib, c, B=-1) == SHAPE
    assert call(lib, c, T=-1) == SHAPE
    assert call(lib, c, lens=None) == ARG
    assert call(lib, c, offsets=None) == ARG
    assert call(lib, c, offsets=0x100002) == ALIGN
    assert call(lib, c, lens=0x100002) == ALIGN
    assert call(lib, c, T=0) == OK and call(lib, c, B=0) == OK
    assert call(lib, _cache(kind=1), T=0) == OK


def test_bad_rows(lib):
    c = _cache()
    for kw in (dict(kt=100), dict(kh=4), dict(vt=-128), dict(vh=-64), dict(k=0x100008),
               dict(v=0x100002)):
        assert _write(lib, c, **kw) == ALIGN, kw
    assert _write(lib, c, k=None) == ARG and _write(lib, c, v=None) == ARG
    assert _read(lib, c, k=None) == ARG and _read(lib, c, v=0x100008) == ALIGN
    for kw in (dict(qt=4), dict(qh=-64), dict(q=0x100008), dict(o=0x100008), dict(lse=0x100004)):
        assert _prefill(lib, c, **kw) == ALIGN, kw


def test_bad_attention_arguments(lib):
    for call, cache, unit in ((_prefill, _cache(), 128), (_decode, _cache(1), 64)):
        assert call(lib, cache, Hq=3) == SHAPE
        assert call(lib, cache, Hq=-4) == SHAPE
        assert call(lib, cache, msl=8 * 16 + 1) == SHAPE
        assert call(lib, cache, msl=-1) == SHAPE
        for split in (0, -unit, unit // 2, unit + 16):
            assert call(lib, cache, split=split) == ARG, split
        assert call(lib, cache, scale=float("nan")) == ARG
        assert call(lib, cache, mask=3) == ARG
        assert call(lib, cache, mask=2) == ARG                    # window without params
        mp = _lib.MaskParams(-1, None, 0)
        assert call(lib, cache, mask=2, mp=ctypes.byref(mp)) == ARG
        assert call(lib, cache, score=4) == ARG                   # no dropout
        assert call(lib, cache, score=2) == ARG
        for c in (0.0, -1.0, float("inf"), float("nan")):
            sp = _lib.ScoreParams(c)
            assert call(lib, cache, score=2, sp=ctypes.byref(sp)) == ARG, c
        for name in ("q", "o", "lse", "lens"):
            assert call(lib, cache, **{name: None}) == ARG, name
        assert call(lib, cache, msl=128, split=unit, Hq=0) == OK
    c = _cache(maxp=64)
    assert _prefill(lib, c, new=-1) == SHAPE
    assert _prefill(lib, c, msl=1000, ws=None) == WORKSPACE
    assert _prefill(lib, c, msl=1000, wsb=100) == WORKSPACE
    assert _prefill(lib, c, msl=1000, ws=0x100010) == ALIGN
    c = _cache(1, maxp=64)
    assert _decode(lib, _cache(0)) == ARG                         # a bf16 cache
    assert _decode(lib, c, msl=1000, ws=None) == WORKSPACE
    assert _decode(lib, c, Nq=-1) == SHAPE
    assert _decode(lib, c, B=1 << 20, Nq=1 << 20) == SHAPE
    assert _decode(lib, c, B=0) == OK and _decode(lib, c, Nq=0) == OK


def _round256(x):
    return (x + 255) // 256 * 256


def test_prefill_sizes(lib):
    ws = lib.attn_prefill_workspace_size
    assert ws(100, 8, 128, 4096, 4096) == 0
    assert ws(100, 8, 128, 0, 128) == 0 and ws(0, 8, 128, 4096, 128) == 0
    assert ws(101, 8, 128, 4097, 1024) == _round256(4 * 5 * 808) + _round256(4 * 5 * 808 * 128)
    split = lib.attn_prefill_split_keys
    for kind in (0, 1):
        for args in [(1, 4096, 32, 8, 4096, 32768, 32768, 152), (16, 128, 32, 8, 8, 32768, 16 * 20000, 152),
                     (1, 1, 8, 8, 1, 100, 100, 152), (3, 70000, 8, 1, 70000, 70000, 99999, 0),
                     (2, 2, 8, 1, 1, (1 << 31) - 1, 1 << 32, 152), (64, 64, 32, 8, 1, 8192, 64 * 4352, 152)]:
            keys = split(kind, *args)
            assert keys >= 128 and keys % 128 == 0, args
        # the row tiles of one long chunk fill the SMs: no split
        assert split(kind, 1, 4096, 32, 8, 4096, 32768, 32768, 152) == 32768
        # a few rows over long caches: split
        assert split(kind, 16, 128, 32, 8, 8, 32768, 16 * 20000, 152) < 32768
        assert split(kind, 0, 0, 8, 8, 0, 0, 0, 152) == 128


def test_binding_refuses_cpu_tensors():
    """CPU tensors never reach the library, also where CUDA was never initialised."""
    import torch

    import exact_io_aware_13_gb300 as ea
    bf = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ea.cache_write(rows, rows, bf, bf, i32(1, 4), i32(2), i32(1))
    with pytest.raises(ValueError):
        ea.cache_read(bf, bf, i32(1, 4), i32(2), i32(1), 3)
    with pytest.raises(ValueError):
        ea.prefill_paged(rows, bf, bf, i32(1, 4), i32(2), i32(1))
    with pytest.raises(ValueError):
        ea.decode_paged(rows[None], bf, bf, i32(1, 4), i32(1))


@pytest.mark.parametrize("kind", [0, 1])
def test_pools_without_pages(lib, kind):
    """A pool of no pages has empty tensors, whose pointers are null: calls without rows are
    no-ops over it, calls with rows are refused, for both kinds alike."""
    c = _cache(kind, pages=0, kc=None, vc=None, exp=None)
    for call in CALLS:
        assert call(lib, c, T=0) == OK and call(lib, c, B=0) == OK, call
        assert call(lib, c) == ARG, call
    if kind == 1:
        assert _decode(lib, c, B=0) == OK and _decode(lib, c, Nq=0) == OK
        assert _decode(lib, c) == ARG
