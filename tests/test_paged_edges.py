"""GPU parity of the paged attention calls at the edges of their range. Bounds as in
test_paged.py, with what a test adds to them stated there."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from tests.paged_inputs import Batch
from tests.test_paged import check_attention, oracle, run_prefill
from workloads import MASK_CAUSAL, MASK_NONE, MASK_SLIDING_WINDOW

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def _put(w, b, t, k=None, v=None):
    """Replaces tokens t of sequence b in the e4m3 cache by rows k, v [len(t), d], the same in
    every kv head."""
    t = np.atleast_1d(t)
    pages, slots = w.table[b, t // w.page], t % w.page
    for i, (cache, x) in enumerate(((w.k_cache, k), (w.v_cache, v))):
        codes, e = P.encode(np.broadcast_to(np.asarray(x, dtype=np.float64), (len(t), w.d)))
        cache[pages, :, slots] = torch.from_numpy(codes)[:, None].expand(-1, w.Hkv, -1)
        w.kv_exp[pages, :, slots, i] = torch.from_numpy(e)[:, None].expand(-1, w.Hkv)


# ------------------------------------------------------------------ V scales far apart
def _light_tail(n, Hq, where, sink):
    """A sink key with V of magnitude `sink`, thousands of tail keys of 2^-20 of its weight that
    carry the output, and one token whose V is 2^15 times theirs: nearly no weight (light), or
    just below the window of every row (masked). The tail keeps its share.

    P holds weights down to 2^-17 of the largest in fp16's 11 bits, and those below in steps of
    2^-27 of it: half a step for each of the L tail keys of at most 1.25 comes beside the
    module's bound (the token that stands out weighs less than 2^-90)."""
    d, L, s0 = 64, 3000, 20.5 * np.log(2.0)
    w = Batch([n], [L], Hq=Hq, Hkv=1, d=d, page=16, kind="e4m3", seed=70)
    q = np.sign(np.random.default_rng(70).standard_normal(d))
    w.q[:] = torch.from_numpy(q).to(torch.bfloat16)
    lo = 100 if where == "masked" else 0          # lowest key that the first row sees
    rng = np.random.default_rng(71)
    _put(w, 0, np.arange(L), k=0.0, v=1.0 + 0.25 * rng.random((L, d)))
    _put(w, 0, lo + n + 1, k=q * (s0 / 8.0), v=sink * rng.standard_normal(d))  # score s0
    big = 2.0 ** 15 * (1.0 + rng.random(d))
    if where == "light":
        _put(w, 0, 0, k=q * -8.0, v=big)                          # score -64
        kw = dict(mask=MASK_NONE)
    else:
        _put(w, 0, lo - 1, k=0.0, v=big)
        kw = dict(mask=MASK_SLIDING_WINDOW, window=L - n - lo + 1)
    o_ref, l_ref, mag = oracle(w, **kw)
    more = 2.0 ** -28 * L * 1.25 / 2.0 ** -8       # as a part of A, which the bound takes 2^-8 of
    for split in (1 << 20, 1024):
        o, lse = run_prefill(w, split=split, **kw)
        assert _ea().device_status() == 0
        check_attention(o, lse, (o_ref, l_ref, mag + more), f"{where} {split}")


@pytest.mark.parametrize("where", ["light", "masked"])
@pytest.mark.parametrize("n,Hq", [(1, 1), (1, 8), (4, 4), (3, 8), (4, 8)])
def test_light_tail_beside_a_large_value(n, Hq, where):
    """Row kernel; the sink's scale lies 2^25 below the largest."""
    _light_tail(n, Hq, where, 2.0 ** -10)


@pytest.mark.parametrize("where", ["light", "masked"])
@pytest.mark.parametrize("n,Hq", [(33, 1), (80, 4)])
def test_light_tail_beside_a_large_value_in_tiles(n, Hq, where):
    """Tile kernel, inside the 2^24 between scales that it is stated for: 2^21 here, codes from 1
    on are exact there. (At 2^25 the factor of the sink's row, 2^-25, is half of fp16's smallest
    number and rounds to 0: that row is lost.)"""
    _light_tail(n, Hq, where, 2.0 ** -6)


@pytest.mark.parametrize("G", [2, 4, 6, 8])
def test_scales_far_apart_in_few_rows(G):
    """K and V scales that differ by many powers of two, zero rows among them, in ragged chunks
    of up to four tokens and in decode with three (8 to 32 rows per kv head)."""
    new, lens = [4, 0, 1, 3, 4], [300, 9, 500, 37, 1300]
    for chunks in (True, False):
        w = Batch(new if chunks else [3] * 5, lens, Hq=2 * G, Hkv=2, d=128, kind="e4m3", page=16,
                  seed=76 + G, k_scale=0.02)
        rng = np.random.default_rng(76)
        owned = w.kv_exp.numpy() != 255
        shift = rng.integers(-12, 3, size=w.kv_exp.shape)
        w.kv_exp = torch.from_numpy(np.where(owned, np.clip(w.kv_exp.numpy().astype(int) + shift, 0, 254),
                                             255).astype(np.uint8))
        for b, t in ((0, 3), (0, 298), (2, 0), (2, 130), (4, 1299)):
            _put(w, b, t, k=0.0, v=0.0)
        for split, mask in ((1 << 20, MASK_CAUSAL), (256, MASK_NONE), (128, MASK_SLIDING_WINDOW)):
            kw = dict(mask=mask, window=90)
            if chunks:
                o, lse = run_prefill(w, split=split, max_new=4, **kw)
            else:
                c = w.cuda()
                q = c["q"].reshape(w.B, 3, w.Hq, w.d).transpose(1, 2).contiguous()
                o, lse = _ea().decode_paged(q, c["k_cache"], c["v_cache"], c["table"], c["seq_lens"],
                                            split_keys=split, mask_kind=mask, window=90,
                                            kv_exp=c["kv_exp"])
                o, lse = o.transpose(1, 2).reshape(-1, w.Hq, w.d), lse.transpose(1, 2).reshape(-1, w.Hq)
            assert _ea().device_status() == 0
            check_attention(o, lse, oracle(w, **kw), f"chunks {chunks} split {split} mask {mask}")


# ------------------------------------------------------------------ pages that are gone
def _free_behind(w, window, how):
    """The page table after the pages that lie wholly below every row's window were freed:
    their entries are -1, or belong to someone whose page is NaN all over."""
    table = w.table.copy()
    owned = set(w.table[w.table >= 0].tolist())
    nan_page = next(p for p in range(w.pages) if p not in owned)   # Batch fills it with NaN
    freed = 0
    for b, (n, L) in enumerate(zip(w.new, w.lens)):
        if n == 0:
            continue
        gone = max(0, L - n - window + 1) // w.page
        table[b, :gone] = -1 if how == "gone" else nan_page
        freed += gone
    assert freed > 0
    return torch.from_numpy(table).cuda()


@pytest.mark.parametrize("how", ["gone", "another's"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 192])
@pytest.mark.parametrize("n,Hq", [(1, 2), (4, 8), (6, 8), (40, 4), (200, 2), (300, 2)])
def test_window_over_freed_pages(n, Hq, page, kind, how):
    """Pages wholly below the windows of all of a call's rows are never followed."""
    for window in (5, 70, 333):
        w = Batch([n, 0, n], [n + 1000, 40, n + 417], Hq=Hq, Hkv=2, d=64, page=page, kind=kind, seed=72)
        ref = oracle(w, MASK_SLIDING_WINDOW, window)
        c = w.cuda()
        c["table"] = _free_behind(w, window, how)
        for split in (128, 1 << 20):
            o, lse = run_prefill(w, c, split=split, mask=MASK_SLIDING_WINDOW, window=window, max_new=n)
            assert _ea().device_status() == 0, (window, split)
            check_attention(o, lse, ref, f"window {window} split {split}")


def _decode_over_freed_pages(nq, Hq, page, kind, how):
    for window in (5, 70, 333):
        w = Batch([nq] * 3, [1000, 400, 777], Hq=Hq, Hkv=2, d=128, page=page, kind=kind, seed=73)
        ref = oracle(w, MASK_SLIDING_WINDOW, window)
        c = w.cuda()
        q = c["q"].reshape(w.B, nq, Hq, w.d).transpose(1, 2).contiguous()
        table = _free_behind(w, window, how)
        for split in (64, 256, 1 << 20):
            o, lse = _ea().decode_paged(q, c["k_cache"], c["v_cache"], table, c["seq_lens"],
                                        split_keys=split, mask_kind=MASK_SLIDING_WINDOW,
                                        window=window, kv_exp=c["kv_exp"])
            assert _ea().device_status() == 0, (window, split)
            check_attention(o.transpose(1, 2).reshape(-1, Hq, w.d),
                            lse.transpose(1, 2).reshape(-1, Hq), ref, f"window {window} split {split}")


@pytest.mark.parametrize("how", ["gone", "another's"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 192])
@pytest.mark.parametrize("nq,Hq", [(1, 8), (3, 16), (9, 16)])
def test_decode_e4m3_window_over_freed_pages(nq, Hq, page, how):
    _decode_over_freed_pages(nq, Hq, page, "e4m3", how)


@pytest.mark.parametrize("how", ["gone", "another's"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 192])
@pytest.mark.parametrize("nq,Hq", [(1, 8), (3, 16), (9, 16), (9, 8)])
def test_decode_bf16_window_over_freed_pages(nq, Hq, page, how):
    _decode_over_freed_pages(nq, Hq, page, "bf16", how)


# ------------------------------------------------------------------ V near the top of the range
@pytest.mark.parametrize("split", [128, 1024, 1 << 20])
@pytest.mark.parametrize("n,Hq", [(1, 2), (4, 4), (4, 8), (33, 2), (70, 1), (300, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_values_near_the_top_of_the_range(n, Hq, d, split):
    """V of one sign up to 1.75 * 2^126 whose weight is spread over every key: the unnormalised
    sums pass fp32's range, the results do not."""
    w = Batch([n], [1500], Hq=Hq, Hkv=1, d=d, page=16, kind="e4m3", seed=74)
    owned = w.kv_exp[..., 1] != 255
    w.v_cache = (w.v_cache & 0x0F) | 0x70                        # 128 .. 448 (no NaN code), positive
    w.v_cache = torch.where(w.v_cache == 0x7F, torch.full_like(w.v_cache, 0x7E), w.v_cache)
    w.kv_exp[..., 1] = torch.where(owned, torch.full_like(w.kv_exp[..., 1], 127 + 118), w.kv_exp[..., 1])
    for mask in (MASK_NONE, MASK_CAUSAL):
        o, lse = run_prefill(w, split=split, mask=mask, max_new=n)
        assert _ea().device_status() == 0
        check_attention(o, lse, oracle(w, mask), f"mask {mask}")


@pytest.mark.parametrize("split", [64, 256, 1 << 20])
def test_decode_values_near_the_top_of_the_range(split):
    w = Batch([1, 1], [20000, 700], Hq=4, Hkv=1, d=128, page=64, kind="e4m3", seed=77)
    w.v_cache, w.kv_exp[..., 1] = torch.full_like(w.v_cache, 0x7E), 127 + 118     # 448 * 2^118
    c = w.cuda()
    o, lse = _ea().decode_paged(c["q"][:, :, None].contiguous(), c["k_cache"], c["v_cache"], c["table"],
                                c["seq_lens"], split_keys=split, kv_exp=c["kv_exp"])
    assert _ea().device_status() == 0
    check_attention(o[:, :, 0], lse[:, :, 0], oracle(w, MASK_NONE), f"split {split}")


@pytest.mark.parametrize("split", [128, 1 << 20])
@pytest.mark.parametrize("n,Hq", [(1, 2), (4, 8), (70, 1), (300, 2)])
def test_values_near_the_bottom_of_the_range(n, Hq, split):
    """V of one sign about 2^-118 whose weight is spread over every key: O is a normal number
    of bf16, and keeps its bits (the module's 1e-6 put aside by scaling both sides)."""
    w = Batch([n], [1500], Hq=Hq, Hkv=1, d=64, page=16, kind="e4m3", seed=78)
    owned = w.kv_exp[..., 1] != 255
    w.v_cache = (w.v_cache & 0x0F) | 0x60                        # 32 .. 120, positive
    w.kv_exp[..., 1] = torch.where(owned, torch.full_like(w.kv_exp[..., 1], 4), w.kv_exp[..., 1])
    o, lse = run_prefill(w, split=split, mask=MASK_NONE, max_new=n)
    o_ref, l_ref, mag = oracle(w, MASK_NONE)
    s = 2.0 ** 118
    check_attention(o.double() * s, lse, (o_ref * s, l_ref, mag * s), f"split {split}")


# ------------------------------------------------------------------ pools without pages
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_over_a_pool_without_pages(kind):
    """Nothing is cached and no page exists: rows without keys, on both kernels' sizes."""
    ea = _ea()
    t, e = (torch.bfloat16, None) if kind == "bf16" else (torch.uint8, torch.empty(0, 2, 16, 2, dtype=torch.uint8))
    e = None if e is None else e.cuda()
    cache = torch.empty(0, 2, 16, 64, dtype=t, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    for n in (1, 50):
        q = torch.ones(2 * n, 4, 64, dtype=torch.bfloat16, device="cuda")
        o, lse = ea.prefill_paged(q, cache, cache, table, i32(0, n, 2 * n), i32(0, 0), kv_exp=e)
        assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    o, lse = ea.decode_paged(q[:2, :, None].contiguous(), cache, cache, table, i32(0, 0), kv_exp=e)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    k = q[:0, :2]
    ea.cache_write(k, k, cache, cache, table, i32(0, 0, 0), i32(0, 0), kv_exp=e)
    assert ea.cache_read(cache, cache, table, i32(0, 0, 0), i32(0, 0), 0, kv_exp=e)[0].shape == (0, 2, 64)
    assert ea.device_status() == 0


# ------------------------------------------------------------------ numbers of decode_paged
def test_decode_takes_the_numbers_that_int_takes():
    """max_seq_len, split_keys and total_kv_tokens as floats and numpy and tensor scalars; the
    form on caller-owned tensors takes no None for them; errors name the entry point."""
    ea = _ea()
    for kind in ("bf16", "e4m3"):
        w = Batch([1, 1], [90, 300], Hq=4, Hkv=2, d=64, kind=kind, seed=75)
        c = w.cuda()
        args = (c["q"].reshape(2, 4, 1, 64), c["k_cache"], c["v_cache"], c["table"], c["seq_lens"])
        want = ea.decode_paged(*args, max_seq_len=304, split_keys=128, total_kv_tokens=390,
                               kv_exp=c["kv_exp"])
        for cast in (float, np.float64, np.int64, torch.tensor, np.float32):
            got = ea.decode_paged(*args, max_seq_len=cast(304), split_keys=cast(128),
                                  total_kv_tokens=cast(390), kv_exp=c["kv_exp"])
            assert all(torch.equal(a, b) for a, b in zip(got, want)), cast
        ea.decode_paged(*args, total_kv_tokens=390.0, kv_exp=c["kv_exp"])
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        good = dict(max_seq_len=304.0, split_keys=128, scale=0.125)
        ea.decode_paged_into(*args, o, lse, ws, kv_exp=c["kv_exp"], **good)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        for name in good:
            with pytest.raises(TypeError):
                ea.decode_paged_into(*args, o, lse, ws, kv_exp=c["kv_exp"], **{**good, name: None})
        with pytest.raises(TypeError):
            ea.decode_paged(*args, max_seq_len=[304], kv_exp=c["kv_exp"])
        with pytest.raises(ValueError):
            ea.decode_paged(*args, max_seq_len=float("nan"), kv_exp=c["kv_exp"])
        with pytest.raises(ea.AttnError, match="^attn_decode_paged" + ("_e4m3" if kind == "e4m3" else "") + ":"):
            ea.decode_paged(*args, split_keys=100, kv_exp=c["kv_exp"])


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_given_stream_does_not_wait_for_the_current_one(kind):
    """Memory that was freed on the current stream while work on it is still queued there is not
    given to a call on another stream, which would finish before that work writes."""
    ea = _ea()
    w = Batch([20, 3, 2], [900, 700, 400], d=128, Hq=8, kind=kind, seed=79)
    c = w.cuda()
    q1 = c["q"][:3].reshape(3, 8, 1, 128)
    cache = (c["k_cache"], c["v_cache"], c["table"])

    def calls(stream):
        out = ea.prefill_paged(c["q"], *cache, c["offsets"], c["seq_lens"], kv_exp=c["kv_exp"],
                               split_keys=256, mask_kind=MASK_CAUSAL, stream=stream)
        out += ea.decode_paged(q1, *cache, c["seq_lens"], kv_exp=c["kv_exp"], split_keys=256, stream=stream)
        return out + ea.cache_read(*cache, c["offsets"], c["seq_lens"], w.T, kv_exp=c["kv_exp"], stream=stream)

    want = calls(None)
    msl = c["table"].shape[1] * w.page
    sizes = [t.nbytes for t in want] + [ea.prefill_workspace_size(T, 8, 128, msl, 256) for T in (w.T, 3)]
    sizes.append(ea.decode_workspace_size(3, 8, w.Hkv, 1, 128, msl, 256))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                  # some 10 ms on the current stream
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    del junk                                       # its fills are still queued
    got = calls(s)
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert ea.device_status() == 0


# ------------------------------------------------------------------ rows of no sequence
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_behind_the_last_sequence_need_no_memory(kind):
    """The C calls with a T beyond offsets[B]: inputs hold the sequences' rows alone, and what
    lies behind the outputs' rows stays."""
    import ctypes

    from exact_io_aware_13_gb300 import _lib
    ea, lib = _ea(), _lib.load()
    w = Batch([4, 0, 9], [30, 7, 9], Hq=4, Hkv=2, d=64, page=16, kind=kind, seed=80)
    c = w.cuda()
    more = w.T + 5000                                     # rows of the calls
    cache = _lib.PagedCache(c["k_cache"].data_ptr(), c["v_cache"].data_ptr(),
                            None if kind == "bf16" else c["kv_exp"].data_ptr(), c["table"].data_ptr(),
                            kind == "e4m3", w.pages, w.Hkv, w.page, w.d, w.table.shape[1])
    ref = ctypes.byref(cache)
    where = (c["offsets"].data_ptr(), c["seq_lens"].data_ptr(), w.B, more)
    stream = torch.cuda.current_stream().cuda_stream
    row = w.Hkv * w.d
    assert lib.attn_cache_write(ref, c["k"].data_ptr(), row, w.d, c["v"].data_ptr(), row, w.d, *where,
                                stream) == 0
    torch.cuda.synchronize()
    want = w.written()
    for got, x in zip((c["k_cache"], c["v_cache"], c["kv_exp"]), want):
        if x is not None:
            view = torch.int16 if x.dtype == torch.bfloat16 else x.dtype
            assert torch.equal(got.cpu().view(view), x.view(view))
    k, v, o = (torch.full((w.T + 3, h, w.d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (2, 2, 4))
    lse = torch.full((w.T + 3, 4), 7.0, device="cuda")
    assert lib.attn_cache_read(ref, k.data_ptr(), v.data_ptr(), *where, stream) == 0
    ws = torch.empty(ea.prefill_workspace_size(more, 4, w.d, 32, 128) + 256, dtype=torch.uint8, device="cuda")
    assert lib.attn_prefill_paged(ref, c["q"].data_ptr(), 4 * w.d, w.d, o.data_ptr(), lse.data_ptr(),
                                  *where, 4, 9, 32, 128, ctypes.c_float(w.d ** -0.5), MASK_CAUSAL, None,
                                  0, None, ws.data_ptr(), ws.numel(), stream) == 0
    torch.cuda.synchronize()
    assert ea.device_status() == 0
    w.k_cache, w.v_cache, w.kv_exp = want
    check_attention(o[:w.T], lse[:w.T], oracle(w), "rows")
    for x in (k, v, o, lse):
        assert bool((x[w.T:] == 7.0).all())
    ex = None if want[2] is None else want[2].numpy()
    kc, vc = (want[0], want[1]) if ex is None else (want[0].numpy(), want[1].numpy())
    for b, n in enumerate(w.new):
        K, V = P.sequence(kc, vc, ex, w.table[b], w.lens[b] - n, w.lens[b])
        for got, x in ((k, K), (v, V)):
            rows = got[w.offsets[b]:w.offsets[b] + n].double().cpu().numpy()
            assert np.array_equal(rows, np.asarray(x, dtype=np.float64))


# ------------------------------------------------------------------ many units
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_more_units_than_sms_over_unequal_caches(kind):
    """Few rows of many sequences in the tile kernel, unsplit by the library's choice, some caches
    a hundred times as long as others; and the same rows in chunks of the library's smallest
    choice."""
    ea = _ea()
    lens = [40 + 37 * i if i % 7 else 4000 + i for i in range(80)]
    w = Batch([5 + i % 4 for i in range(80)], lens, Hq=20, Hkv=2, d=64, page=64, kind=kind, seed=81)
    assert ea.prefill_split_keys(kind == "e4m3", 80, w.T, 20, 2, 8, 4096, sum(lens)) >= 4096
    rows = np.unique(np.concatenate([w.offsets[:-1], w.offsets[1:] - 1]))   # the oracle's share
    for split, mask in ((None, MASK_CAUSAL), (1024, MASK_NONE)):
        o, lse = run_prefill(w, split=split, mask=mask, max_new=8, total_kv_tokens=sum(lens))
        assert ea.device_status() == 0
        check_attention(o, lse, oracle(w, mask, rows=rows), f"split {split}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [255, 257])
def test_merge_on_both_sides_of_its_rule(n, kind):
    """More than eight chunks with just under and just over 2048 rows."""
    w = Batch([n], [1500], Hq=8, Hkv=2, d=128, page=64, kind=kind, seed=82)
    rows = np.arange(0, n, 16)
    o, lse = run_prefill(w, split=128)
    assert _ea().device_status() == 0
    check_attention(o, lse, oracle(w, MASK_CAUSAL, rows=rows), f"rows {8 * n}")
