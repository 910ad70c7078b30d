"""What the paged kernels check before they follow a device input (csrc/paged_index.cuh,
built for the host): spans with bad offsets and lengths, page indices outside the pool, and
the page walk against division. CPU only."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "host", "paged_host.cpp")
CSRC = os.path.join(ROOT, "exact_io_aware_13_gb300", "csrc")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("paged_host") / "paged_host.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-x", "c++", SRC, "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.host_row.restype = ctypes.c_longlong
    return lib


def test_spans(host):
    T, new, msl = 100, 40, 5000
    good = [(0, 0, 0), (0, 40, 5000), (60, 100, 1), (100, 100, 7)]
    bad = [(-1, 3, 10), (5, 4, 10), (61, 101, 10), (0, 41, 10), (0, 1, -1), (0, 1, 5001),
           (-2**31, 2**31 - 1, 0), (2**31 - 1, -2**31, 0), (99, 2**31 - 1, 0)]
    for o0, o1, L in good:
        assert host.host_span_ok(T, new, msl, o0, o1, L), (o0, o1, L)
    for o0, o1, L in bad:
        assert not host.host_span_ok(T, new, msl, o0, o1, L), (o0, o1, L)


def test_rows_stay_inside_the_pool(host):
    for pages, Hkv, ps in [(1, 1, 8), (7, 3, 16), (2**20, 8, 192)]:
        for page in (-2**31, -1, pages, pages + 5, 2**31 - 1):
            assert host.host_row(page, pages, Hkv, ps, 0, 0) == -1
        for page in {0, pages // 2, pages - 1}:
            for head in {0, Hkv - 1}:
                for slot in (0, ps - 1):
                    want = (page * Hkv + head) * ps + slot
                    got = host.host_row(page, pages, Hkv, ps, head, slot)
                    assert got == want and 0 <= got < pages * Hkv * ps


@pytest.mark.parametrize("stride", [64, 128])
@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128, 192, 256, 320, 1024])
def test_walk_is_division(host, stride, ps):
    n = 200
    for key0 in (0, 8, 32, 64, 96, 128, 8 * 123):
        pages, slots = np.zeros(n, dtype=np.int32), np.zeros(n, dtype=np.int32)
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        host.host_walk(key0, stride, ps, n, p(pages), p(slots))
        keys = key0 + stride * np.arange(n)
        assert np.array_equal(pages, keys // ps) and np.array_equal(slots, keys % ps)


@pytest.mark.parametrize("tile", [32, 64, 128])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_skipped_keys_are_the_pieces_below(host, tile, R):
    """In the tile that holds k_lo: every key of a piece that ends at or below k_lo, no other."""
    if R > tile:
        return
    for t0 in (0, tile, 7 * tile, (2**31 - 4096) // tile * tile - tile):
        for k_lo in range(max(0, t0 - 3), t0 + tile):
            want = sum((t0 + k) // R * R + R <= k_lo for k in range(tile))
            assert host.host_skipped_keys(t0, k_lo, R) == want
    assert host.host_skipped_keys(0, 0, R) == 0
