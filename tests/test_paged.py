"""GPU parity of the paged cache: writing and reading tokens (bit for bit against the
oracle's format) and attention of ragged chunks of new tokens (against float64).

Bound of an output element: O is rounded to bf16 once (at most 2^-8 of the value, half a
step) and P once before the P V product (bf16 at worst: 2^-8 of each term, so 2^-8 A with
A = sum_j P |V|). The scores are exact products summed in fp32 (d <= 128 terms of a few
units: below 2^-17 absolute) and scaled; exp2 and the sums add less than 2^-20 relative;
a hardware tanh is off by at most 7.8e-6 c, here c = 7: 5.5e-5. Together these move a
weight, and its row sum, by less than 2^-12 each: 2^-11 A. So
|dO| <= 2^-8 |O| + (2^-8 + 2^-11) A + 1e-6 and |dLSE| <= 2e-4. Where scores are large on
purpose, fp32 sums of d products and the scaling move a score by up to
delta = (d + 4) 2^-24 max_rows sum |q| |k| scale, a weight and its row sum by e^delta each:
2 delta A and delta come on top (`delta` below).
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from tests.paged_inputs import Batch
from workloads import MASK_CAUSAL, MASK_NONE, MASK_SLIDING_WINDOW, SCORE_ALIBI, SCORE_SOFTCAP

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def check_attention(o, lse, ref, what="", delta=0.0):
    o_ref, l_ref, mag = ref
    o, lse = np.asarray(o.float().cpu().numpy(), dtype=np.float64), lse.cpu().numpy()
    rows = ~np.isnan(l_ref)
    o, lse, o_ref, l_ref, mag = o[rows], lse[rows], o_ref[rows], l_ref[rows], mag[rows]
    empty = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(lse), empty), what
    assert np.all(o[empty] == 0), what
    assert np.all(np.isfinite(o)), what
    bound = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -8 + 2.0 ** -11 + 2 * delta) * mag + 1e-6
    over = np.abs(o - o_ref) / bound
    assert over.max(initial=0.0) <= 1.0, f"{what}: |dO| {over.max()} of its bound"
    err = np.abs(lse[~empty] - l_ref[~empty]).max(initial=0.0)
    assert err <= 2e-4 + delta, f"{what}: |dLSE| {err}"


def run_prefill(w, dev=None, *, mask=MASK_CAUSAL, window=0, score=0, softcap=7.0, split=None, **kw):
    ea = _ea()
    c = dev or w.cuda()
    o, lse = ea.prefill_paged(c["q"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                              c["seq_lens"], kv_exp=c["kv_exp"], split_keys=split,
                              mask_kind=mask, window=window, score_kind=score,
                              softcap=softcap if score & SCORE_SOFTCAP else 0.0, **kw)
    torch.cuda.synchronize()
    return o, lse


def oracle(w, mask=MASK_CAUSAL, window=0, score=0, softcap=7.0, rows=None):
    return P.chunk_forward(w.q, w.k_cache, w.v_cache, w.kv_exp, w.table, w.offsets, w.lens,
                           w.d ** -0.5, mask, window, score, softcap, rows=rows)


def score_delta(w):
    """delta of the module's bound for this batch."""
    top = 0.0
    for b, L in enumerate(w.lens):
        K, _ = P.sequence(w.k_cache, w.v_cache, w.kv_exp, w.table[b], 0, L)
        q = np.abs(w.q[w.offsets[b]:w.offsets[b + 1]].double().numpy())
        for h in range(w.Hq):
            top = max(top, (q[:, h] @ np.abs(K[:, h // (w.Hq // w.Hkv)]).T).max(initial=0.0))
    return (w.d + 4) * 2.0 ** -24 * top * w.d ** -0.5


def parity(w, what="", split=None, rows=None, delta=0.0, **kw):
    o, lse = run_prefill(w, split=split, **kw)
    assert _ea().device_status() == 0
    check_attention(o, lse, oracle(w, rows=rows, **kw), what, delta)


# ------------------------------------------------------------------ write and read
def _write(w, c):
    _ea().cache_write(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                      c["seq_lens"], kv_exp=c["kv_exp"])
    torch.cuda.synchronize()


def _same_cache(c, want):
    for got, ref in zip((c["k_cache"], c["v_cache"], c["kv_exp"]), want):
        if ref is not None:
            view = torch.int16 if ref.dtype == torch.bfloat16 else ref.dtype
            assert torch.equal(got.cpu().view(view), ref.view(view))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 64, 192])
def test_write_and_read(kind, d, page):
    w = Batch([3, 0, 1, 70, 0], [9, 5, 1, 200, 0], d=d, page=page, kind=kind, Hkv=3, Hq=3,
              seed=page + d, spare_rows=5)
    c = w.cuda()
    _write(w, c)
    want = w.written()
    _same_cache(c, want)
    # reading the same rows gives back what the cache holds; rows behind the last sequence stay
    ea = _ea()
    k = torch.full((w.T, w.Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 9.0)
    ea.cache_read_into(c["k_cache"], c["v_cache"], c["table"], c["offsets"], c["seq_lens"], k, v,
                       kv_exp=c["kv_exp"])
    assert ea.device_status() == 0
    ex = None if want[2] is None else want[2].numpy()
    kc, vc = (want[0], want[1]) if ex is None else (want[0].numpy(), want[1].numpy())
    for b, n in enumerate(w.new):
        K, V = P.sequence(kc, vc, ex, w.table[b], w.lens[b] - n, w.lens[b])
        o = int(w.offsets[b])
        assert np.array_equal(k[o:o + n].double().cpu().numpy(), np.asarray(K, dtype=np.float64))
        assert np.array_equal(v[o:o + n].double().cpu().numpy(), np.asarray(V, dtype=np.float64))
    assert bool((k[w.rows:] == 7.0).all()) and bool((v[w.rows:] == 9.0).all())


@pytest.mark.parametrize("Hkv", [1, 2, 5, 8, 33])
def test_write_head_counts(Hkv):
    for d in (64, 128):
        w = Batch([2, 130], [40, 131], d=d, Hkv=Hkv, Hq=Hkv, kind="e4m3", seed=Hkv)
        c = w.cuda()
        _write(w, c)
        _same_cache(c, w.written())


@pytest.mark.parametrize("kind", KINDS)
def test_write_strided_rows(kind):
    """k and v as slices of fused projection rows, and as head-major tensors."""
    w = Batch([4, 11], [30, 11], d=64, kind=kind, seed=5)
    want = w.written()
    c = w.cuda()
    fused = torch.cat([c["q"], c["k"], c["v"]], dim=1)
    c["k"], c["v"] = fused[:, w.Hq:w.Hq + w.Hkv], fused[:, w.Hq + w.Hkv:]
    _write(w, c)
    _same_cache(c, want)
    c = w.cuda()
    c["k"] = c["k"].transpose(0, 1).contiguous().transpose(0, 1)
    c["v"] = c["v"].transpose(0, 1).contiguous().transpose(0, 1)
    _write(w, c)
    _same_cache(c, want)


def test_write_special_values():
    """Zero rows, subnormals, the largest bf16, values at a scale's edge, ties, infinities
    and NaN: codes and exponents equal the oracle's bit for bit."""
    w = Batch([12], [12], d=64, Hkv=1, Hq=1, kind="e4m3", seed=6)
    x = torch.zeros(12, 1, 64)
    x[1, 0, 0] = -0.0
    x[2, 0, :3] = torch.tensor([448.0, 447.0, 0.001])
    x[3, 0, :3] = torch.tensor([450.0, 1.0, -2.0])
    x[4, 0, :2] = torch.tensor([3.3895e38, 1.0])
    x[5, 0, :2] = torch.tensor([2.0 ** -133, 2.0 ** -130])
    x[6, 0, :2] = torch.tensor([2.0 ** -126, -2.0 ** -120])
    x[7, 0, :3] = torch.tensor([float("inf"), 3.0, -float("inf")])
    x[8, 0, :3] = torch.tensor([float("nan"), 100.0, 0.5])
    x[9, 0, :] = float("inf")
    x[10, 0] = torch.linspace(-448, 448, 64)
    x[11, 0] = torch.arange(64) + 200.0     # codes of step 16: ties go to even
    w.k = x.to(torch.bfloat16)
    w.v = torch.flip(w.k, dims=[2])
    c = w.cuda()
    _write(w, c)
    want = w.written()
    # a NaN's sign is not defined
    for got, ref in zip((c["k_cache"].cpu(), c["v_cache"].cpu()), want):
        nan = (ref & 127) == 127
        assert torch.equal((got & 127) == 127, nan)
        assert torch.equal(got[~nan], ref[~nan])
    assert torch.equal(c["kv_exp"].cpu(), want[2])


@pytest.mark.parametrize("kind", KINDS)
def test_bad_device_inputs_of_write_and_read(kind):
    """Positions below 0, offsets that do not rise or pass T, lengths above the table's
    capacity and pages outside the pool are reported; nothing outside the cache is written
    and the sequences with good inputs are served."""
    ea = _ea()
    for what in ("position", "offsets", "total", "length", "page", "first"):
        w = Batch([4, 4], [20, 30], kind=kind, seed=7)
        c = w.cuda()
        before = [None if c[n] is None else c[n].clone() for n in ("k_cache", "v_cache", "kv_exp")]
        if what == "position":
            c["seq_lens"][1] = 2
        elif what == "offsets":
            c["offsets"][1] = 9
        elif what == "total":
            c["offsets"][2] = w.T + 1
        elif what == "length":
            c["seq_lens"][1] = 10_000
        elif what == "page":
            c["table"][1] = w.pages + 3
        else:
            c["offsets"][0] = 1
        _write(w, c)
        assert ea.device_status() == 8, what
        ea.cache_read(c["k_cache"], c["v_cache"], c["table"], c["offsets"], c["seq_lens"], w.T,
                      kv_exp=c["kv_exp"])
        assert ea.device_status() == 8, what
        if what in ("length", "page", "total"):   # sequence 0 is good: its slots, no others
            only = Batch([4, 0], [20, 30], kind=kind, seed=7)
            only.k, only.v = w.k, w.v
            only.k_cache, only.v_cache, only.kv_exp = (None if t is None else t.cpu() for t in before)
            _same_cache(c, only.written())
    assert ea.device_status() == 0


# ------------------------------------------------------------------ chunk attention
MIX = dict(new=[1, 0, 7, 33, 5, 1, 2], lens=[1, 4, 64, 200, 3, 700, 0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("split", [128, 256, None])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 192])
def test_prefill_pages_and_splits(kind, page, split):
    """Ragged chunks (0 and 1 tokens, more new tokens than cached, an empty cache) over
    poisoned pools."""
    w = Batch(**MIX, page=page, kind=kind, seed=11)
    parity(w, f"page {page} split {split} {kind}", split=split)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", [0, SCORE_ALIBI, SCORE_SOFTCAP, SCORE_ALIBI | SCORE_SOFTCAP])
@pytest.mark.parametrize("mask,window", [(MASK_NONE, 0), (MASK_CAUSAL, 0), (MASK_SLIDING_WINDOW, 60),
                                         (MASK_SLIDING_WINDOW, 1), (MASK_SLIDING_WINDOW, 0),
                                         (MASK_SLIDING_WINDOW, (1 << 31) - 1)])
def test_prefill_masks_and_scores(kind, mask, window, score):
    for d, split in ((64, 128), (128, None)):
        w = Batch(**MIX, d=d, kind=kind, seed=12)
        parity(w, f"mask {mask} W {window} score {score} d {d}", split=split, mask=mask,
               window=window, score=score)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (6, 2), (7, 7), (16, 2), (17, 1), (40, 1), (150, 1),
                                    (300, 1)])
def test_prefill_head_groups(kind, Hq, Hkv):
    """Groups of 1 to 300 query heads, so that a row tile ends inside a token."""
    w = Batch([3, 1, 61], [150, 129, 61], Hq=Hq, Hkv=Hkv, d=128, page=32, kind=kind, seed=Hq)
    parity(w, f"Hq {Hq} Hkv {Hkv}")
    parity(w, f"Hq {Hq} Hkv {Hkv} split", split=128, mask=MASK_NONE)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 127, 128, 129, 255, 256, 257, 600])
def test_prefill_row_tiles(kind, n):
    """Chunk lengths around the row tiles, alone and behind a cached prefix."""
    w = Batch([n, n], [n, n + 131], Hq=2, Hkv=2, d=64, page=16, kind=kind, seed=n)
    parity(w, f"n {n}")
    w = Batch([n], [n + 1], Hq=1, Hkv=1, d=128, page=64, kind=kind, seed=n)
    parity(w, f"n {n} window", mask=MASK_SLIDING_WINDOW, window=100)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_many_sequences(kind):
    """More sequences than a warp has lanes, most of them short or empty."""
    rng = np.random.default_rng(13)
    new = rng.integers(0, 6, size=75).tolist()
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 90, size=75))]
    w = Batch(new, lens, kind=kind, page=8, seed=13)
    parity(w, "75 sequences")
    parity(w, "75 sequences, max_new", split=128, mask=MASK_NONE)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_large_scores_and_a_sink(kind):
    """Scores of several hundred (a running maximum that jumps at every tile), and one key
    that takes nearly all the weight while the tail of many keys still counts."""
    w = Batch([40, 3], [900, 700], d=64, kind=kind, seed=14, k_scale=40.0)
    parity(w, "large scores", mask=MASK_NONE, delta=score_delta(w))
    w = Batch([4], [3000], Hq=1, Hkv=1, d=64, kind=kind, seed=15, page=64, k_scale=0.01)
    kc = w.k_cache if kind == "bf16" else None
    if kc is not None:
        kc[w.table[0, 0], 0, 0] = w.q[0, 0] * 12.0
    else:
        codes, e = P.encode((w.q[0, 0].double() * 12.0).numpy())
        w.k_cache[w.table[0, 0], 0, 0] = torch.from_numpy(codes)
        w.kv_exp[w.table[0, 0], 0, 0, 0] = int(e)
    parity(w, "sink", mask=MASK_NONE)


def test_prefill_scales_far_apart():
    """Tokens whose K and V scales differ by many powers of two, zero rows among them."""
    w = Batch([9, 200], [300, 500], d=128, kind="e4m3", page=16, seed=16, k_scale=0.02)
    rng = np.random.default_rng(16)
    owned = w.kv_exp.numpy() != 255
    shift = rng.integers(-12, 3, size=w.kv_exp.shape)
    w.kv_exp = torch.from_numpy(np.where(owned, np.clip(w.kv_exp.numpy().astype(int) + shift, 0, 254),
                                         255).astype(np.uint8))
    for b, t in ((0, 3), (0, 298), (1, 0), (1, 130), (1, 499)):   # zero rows: byte 0, codes 0
        page, slot = w.table[b, t // w.page], t % w.page
        w.k_cache[page, :, slot] = 0
        w.v_cache[page, :, slot] = 0
        w.kv_exp[page, :, slot] = 0
    parity(w, "scales")
    parity(w, "scales split", split=128, mask=MASK_NONE, score=SCORE_ALIBI)
    # a whole cache of zero rows: O = 0, uniform weights
    w = Batch([5], [200], d=64, kind="e4m3", seed=17)
    w.k_cache[:], w.v_cache[:] = 0, 0
    w.kv_exp[:] = 0
    o, lse = run_prefill(w, mask=MASK_NONE)
    assert bool((o == 0).all())
    np.testing.assert_allclose(lse.cpu().numpy(), np.log(200.0), atol=1e-5)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_query_magnitudes(kind):
    """Query rows from 2^-40 to 2^8, a zero row among them."""
    w = Batch([30], [160], d=128, kind=kind, seed=18, k_scale=0.05)
    e = torch.linspace(-40, 8, 30).round()
    w.q = (w.q.float() * torch.exp2(e)[:, None, None]).to(torch.bfloat16)
    w.q[7] = 0
    parity(w, "query magnitudes", mask=MASK_NONE, delta=score_delta(w))


def _nan_key(w, b, t):
    """Makes the K row of token t of sequence b NaN, in every kv head."""
    page, slot = w.table[b, t // w.page], t % w.page
    if w.kind == "bf16":
        w.k_cache[page, :, slot] = float("nan")
    else:
        w.k_cache[page, :, slot] = 127


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("split", [128, 1 << 20])
@pytest.mark.parametrize("n,Hq", [(1, 2), (4, 4), (16, 4), (20, 4), (140, 4), (300, 2)])
def test_nan_rows_stay_rows(n, Hq, split, kind):
    """NaN in a query row, and in the K row of a new token under a causal mask: the rows that
    see it become NaN in O and lse, the others are what they are without it. The lengths put
    the NaN key into the first, a middle and the last chunk and tile, alone there too."""
    for mask, at in ((MASK_CAUSAL, 0.5), (MASK_CAUSAL, 0.0), (MASK_NONE, 1.0), (MASK_SLIDING_WINDOW, 0.5)):
        w = Batch([n, n], [1500, n + 130], Hq=Hq, Hkv=2, d=64, page=16, kind=kind, seed=19)
        o_ref, l_ref, mag = oracle(w, mask, 5)
        bad = np.zeros((w.T, Hq), dtype=bool)
        w.q[n // 2, 1] = float("nan")
        bad[n // 2, 1] = True
        for b, L in enumerate(w.lens):
            key = L - n + min(int(at * n), n - 1)
            _nan_key(w, b, key)
            for i in range(n):
                pos = L - n + i
                seen = (mask == MASK_NONE or key <= pos) and (mask != MASK_SLIDING_WINDOW or pos - key < 5)
                bad[b * n + i] |= seen
        o, lse = run_prefill(w, split=split, mask=mask, window=5)
        assert _ea().device_status() == 0
        got = np.isnan(lse.cpu().numpy())
        assert np.array_equal(got, bad), (mask, at, np.argwhere(got != bad)[:8])
        assert np.array_equal(np.isnan(o.float().cpu().numpy()).all(-1), bad), (mask, at)
        l_ref[bad] = np.nan
        check_attention(o, lse, (o_ref, l_ref, mag), f"NaN beside {mask} {at}")


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_strided_queries_and_spare_rows(kind):
    """q as a slice of fused rows and head-major; rows behind the last sequence stay."""
    ea = _ea()
    w = Batch([20, 3], [90, 200], d=64, kind=kind, seed=19, spare_rows=4)
    c = w.cuda()
    base, base_lse = run_prefill(w, c)
    fused = torch.cat([c["q"], c["k"], c["v"]], dim=1)
    views = [fused[:, :w.Hq], c["q"].transpose(0, 1).contiguous().transpose(0, 1)]
    for q in views:
        o = torch.full((w.T, w.Hq, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((w.T, w.Hq), 5.0, device="cuda")
        ws = torch.empty(ea.prefill_workspace_size(w.T, w.Hq, 64, 208, 128), dtype=torch.uint8,
                         device="cuda")
        ea.prefill_paged_into(q, c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                              c["seq_lens"], o, lse, ws, max_new=20, max_seq_len=208,
                              split_keys=128, scale=0.125, kv_exp=c["kv_exp"],
                              mask_kind=MASK_CAUSAL)
        check_attention(o[:w.rows], lse[:w.rows], [x[:w.rows] for x in oracle(w)], "strided")
        assert bool((o[w.rows:] == 3.0).all()) and bool((lse[w.rows:] == 5.0).all())
    check_attention(base[:w.rows], base_lse[:w.rows], [x[:w.rows] for x in oracle(w)], "contiguous")


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_is_deterministic_and_runs_on_its_stream_and_in_graphs(kind):
    ea = _ea()
    w = Batch([20, 3, 150], [90, 700, 400], d=128, kind=kind, seed=20)
    c = w.cuda()
    first, z1 = run_prefill(w, c, split=256)
    again, z2 = run_prefill(w, c, split=256)
    assert torch.equal(first, again) and torch.equal(z1, z2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other, z3 = run_prefill(w, c, split=256)
    assert torch.equal(first, other) and torch.equal(z1, z3)
    # a step in a graph: write the new tokens, attend; replayed on other values and lengths
    msl = c["table"].shape[1] * w.page
    o, lse = torch.empty_like(first), torch.empty_like(z1)
    ws = torch.empty(ea.prefill_workspace_size(w.T, w.Hq, 128, msl, 256), dtype=torch.uint8,
                     device="cuda")

    def step():
        ea.cache_write(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                       c["seq_lens"], kv_exp=c["kv_exp"])
        ea.prefill_paged_into(c["q"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                              c["seq_lens"], o, lse, ws, max_new=150, max_seq_len=msl,
                              split_keys=256, scale=128 ** -0.5, kv_exp=c["kv_exp"],
                              mask_kind=MASK_CAUSAL)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (21, 22):
        w2 = Batch([20, 3, 150], [90, 700, 400], d=128, kind=kind, seed=seed)
        for n in ("q", "k", "v"):
            c[n].copy_(getattr(w2, n))
        g.replay()
        w.q, w.k, w.v = w2.q, w2.k, w2.v
        w.k_cache, w.v_cache, w.kv_exp = w.written()
        torch.cuda.synchronize()
        _same_cache(c, (w.k_cache, w.v_cache, w.kv_exp))
        check_attention(o, lse, oracle(w), "graph")
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_empty_calls(kind):
    ea = _ea()
    w = Batch([0, 0], [5, 0], kind=kind, seed=23)
    o, lse = run_prefill(w)
    assert o.shape == (0, w.Hq, w.d) and lse.shape == (0, w.Hq)
    w = Batch([2, 3], [0, 0], kind=kind, seed=24)   # new tokens and an empty cache
    o, lse = run_prefill(w, mask=MASK_NONE, max_seq_len=0)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    c = w.cuda()
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    ea.cache_write(c["k"], c["v"], c["k_cache"], c["v_cache"], c["table"][:0], z, e,
                   kv_exp=c["kv_exp"])
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_bad_device_inputs(kind):
    ea = _ea()
    for what in ("offsets", "total", "length", "page", "first", "max_new"):
        w = Batch([40, 4], [200, 300], kind=kind, seed=25)
        c = w.cuda()
        kw = {}
        if what == "offsets":
            c["offsets"][1] = 50
        elif what == "total":
            c["offsets"][2] = w.T + 1
        elif what == "length":
            c["seq_lens"][1] = 10_000
        elif what == "page":
            c["table"][1, 2] = w.pages + 3
        elif what == "first":
            c["offsets"][0] = 1
        else:
            kw["max_new"] = 39
        for split in (128, None):
            o, lse = run_prefill(w, c, split=split, **kw)
            assert ea.device_status() == 8, what
        if what in ("length", "page", "total"):
            ref = [x[:40] for x in oracle(w)]
            check_attention(o[:40], lse[:40], ref, what)
    assert ea.device_status() == 0


def test_read_every_scale():
    """Every code under every scale byte: the rounded bf16 of code * 2^(byte - 127)."""
    ea = _ea()
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).reshape(1, 2, 128)
    n = 255
    kc = codes.repeat(n, 1, 1)                       # token t, heads 0 and 1, half the codes each
    pages, page = 16, 16
    cache = torch.zeros(pages, 2, page, 128, dtype=torch.uint8)
    ex = torch.zeros(pages, 2, page, 2, dtype=torch.uint8)
    t = torch.arange(n)
    cache[t // page, :, t % page] = kc
    ex[t // page, :, t % page] = t.to(torch.uint8)[:, None, None].expand(-1, 2, 2)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    k, v = ea.cache_read(cache.cuda(), cache.cuda(), table, i32(0, n), i32(n), n, kv_exp=ex.cuda())
    assert ea.device_status() == 0
    want = torch.from_numpy(P.decode(kc.numpy(), t.to(torch.uint8)[:, None].expand(-1, 2).numpy()))
    want = want.float().to(torch.bfloat16)           # exact in fp32, or beyond its largest number
    for got in (k.cpu(), v.cpu()):
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan].view(torch.int16), want[~nan].view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
def test_caches_past_32_bits(kind):
    """Pages whose byte offsets pass 2^32 (and, for bf16, element offsets too): written, read
    back, attended to and decoded like the same pages at the front of a small pool."""
    ea = _ea()
    w = Batch([200, 1, 3], [300, 700, 3], Hq=8, Hkv=4, d=128, page=64, kind=kind, seed=50)
    c = w.cuda()
    row_bytes = 128 * (2 if kind == "bf16" else 1)
    far = (1 << 32) * 9 // 8 // (row_bytes * 4 * 64)         # first page past 2^32 bytes, and on
    big = dict(c)
    for n in ("k_cache", "v_cache", "kv_exp"):
        if c[n] is not None:
            t = torch.empty((far + w.pages,) + tuple(c[n].shape[1:]), dtype=c[n].dtype, device="cuda")
            t[far:] = c[n]
            big[n] = t
    big["table"] = torch.where(c["table"] >= 0, c["table"] + far, c["table"])
    for x in (c, big):
        _write(w, x)
    for n in ("k_cache", "v_cache", "kv_exp"):
        if c[n] is not None:
            view = torch.int16 if kind == "bf16" else torch.uint8
            assert torch.equal(big[n][far:].view(view), c[n].view(view))
    outs = []
    for x in (c, big):
        kv = ea.cache_read(x["k_cache"], x["v_cache"], x["table"], x["offsets"], x["seq_lens"], w.rows,
                           kv_exp=x["kv_exp"])
        o = run_prefill(w, x, split=128)
        d = ea.decode_paged(x["q"][:3].reshape(3, 8, 1, 128), x["k_cache"], x["v_cache"], x["table"],
                            x["seq_lens"], kv_exp=x["kv_exp"])
        outs.append(kv + o + d)
    torch.cuda.synchronize()
    assert ea.device_status() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_bf16_cache_from_prompt_to_decode():
    """The bf16 path a serving step takes: prompts written, attended to in chunks, then decode
    steps by attn_decode_paged on the cache that cache_write filled."""
    ea = _ea()
    w = Batch([37, 5, 80], [37, 5, 80], Hq=8, Hkv=2, d=128, page=16, seed=51)
    c = w.cuda()
    _write(w, c)
    w.k_cache, w.v_cache, _ = w.written()
    o, lse = run_prefill(w, c)
    check_attention(o, lse, oracle(w), "prompts")
    last = torch.tensor([36, 41, 121], device="cuda")         # the newest token of each sequence
    od, ld = ea.decode_paged(c["q"][last][:, :, None].contiguous(), c["k_cache"], c["v_cache"],
                             c["table"], c["seq_lens"])
    ref = [x[last.cpu().numpy()] for x in oracle(w)]
    check_attention(od[:, :, 0], ld[:, :, 0], ref, "decode on the written cache")
    assert ea.device_status() == 0


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams: each gets the result it gets alone."""
    ea = _ea()
    ws = [Batch([20, 3, 150], [900, 700, 400], d=128, kind=k, seed=52) for k in KINDS]
    cs = [w.cuda() for w in ws]
    alone = [run_prefill(w, c, split=256) for w, c in zip(ws, cs)]
    streams = [torch.cuda.Stream() for _ in ws]
    for _ in range(5):
        outs = []
        for w, c, st in zip(ws, cs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                outs.append(ea.prefill_paged(c["q"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                                             c["seq_lens"], kv_exp=c["kv_exp"], split_keys=256,
                                             mask_kind=MASK_CAUSAL))
        torch.cuda.synchronize()
        for (o, z), (o1, z1) in zip(outs, alone):
            assert torch.equal(o, o1) and torch.equal(z, z1)


@pytest.mark.parametrize("kind", KINDS)
def test_a_given_stream_keeps_the_call_s_tensors(kind):
    """A call on a stream that is not the current one, queued behind other work there: the
    workspace and outputs made for it are not handed out again before it has run."""
    ea = _ea()
    w = Batch([20, 3, 2], [900, 700, 400], d=128, Hq=8, kind=kind, seed=53)
    c = w.cuda()
    q1 = c["q"][:3].reshape(3, 8, 1, 128)
    want = run_prefill(w, c, split=256)
    want_d = ea.decode_paged(q1, c["k_cache"], c["v_cache"], c["table"], c["seq_lens"],
                             kv_exp=c["kv_exp"], split_keys=256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                  # some 10 ms
    got = ea.prefill_paged(c["q"], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                           c["seq_lens"], kv_exp=c["kv_exp"], split_keys=256,
                           mask_kind=MASK_CAUSAL, stream=s)
    got_d = ea.decode_paged(q1, c["k_cache"], c["v_cache"], c["table"], c["seq_lens"],
                            kv_exp=c["kv_exp"], split_keys=256, stream=s)
    msl = c["table"].shape[1] * w.page
    for T in (w.T, 3):                                 # what the allocator would hand out next
        n = ea.prefill_workspace_size(T, 8, 128, msl, 256)
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in zip(got + got_d, want + want_d):
        assert torch.equal(a, b)
    del junk
    assert ea.device_status() == 0


def test_max_new_of_zero_is_reported():
    ea = _ea()
    for kind in KINDS:
        w = Batch([5], [40], Hq=40, Hkv=1, kind=kind, seed=54)
        run_prefill(w, max_new=0)
        assert ea.device_status() == 8


# ------------------------------------------------------------------ decode over e4m3
def run_decode(w, nq, *, mask=MASK_NONE, window=0, score=0, softcap=7.0, split=128, max_seq_len=None):
    ea = _ea()
    c = w.cuda()
    q = c["q"].reshape(w.B, nq, w.Hq, w.d).transpose(1, 2).contiguous()
    o, lse = ea.decode_paged(q, c["k_cache"], c["v_cache"], c["table"], c["seq_lens"],
                             split_keys=split, max_seq_len=max_seq_len, mask_kind=mask,
                             window=window, score_kind=score,
                             softcap=softcap if score & SCORE_SOFTCAP else 0.0, kv_exp=c["kv_exp"])
    torch.cuda.synchronize()
    assert ea.device_status() == 0
    ref = oracle(w, mask, window, score, softcap)
    check_attention(o.transpose(1, 2).reshape(-1, w.Hq, w.d), lse.transpose(1, 2).reshape(-1, w.Hq),
                    ref, f"nq {nq} mask {mask} {window} score {score} split {split}")
    return o, lse


LENS = [0, 1, 63, 64, 65, 200, 700]


@pytest.mark.parametrize("split", [64, 256, 1 << 20])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 192])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_e4m3_pages_and_splits(page, split, d):
    run_decode(Batch([1] * 7, LENS, Hq=8, Hkv=2, d=d, page=page, kind="e4m3", seed=30), 1, split=split)


@pytest.mark.parametrize("score", [0, SCORE_ALIBI, SCORE_SOFTCAP, SCORE_ALIBI | SCORE_SOFTCAP])
@pytest.mark.parametrize("mask,window", [(MASK_NONE, 0), (MASK_CAUSAL, 0), (MASK_SLIDING_WINDOW, 100),
                                         (MASK_SLIDING_WINDOW, 0)])
@pytest.mark.parametrize("nq", [1, 3])
def test_decode_e4m3_masks_and_scores(nq, mask, window, score):
    run_decode(Batch([nq] * 7, LENS, Hq=8, Hkv=2, d=128, kind="e4m3", seed=31 + nq), nq, mask=mask,
               window=window, score=score)


@pytest.mark.parametrize("Hq,Hkv,nq", [(1, 1, 1), (3, 3, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1), (17, 1, 1),
                                       (32, 1, 1), (33, 1, 1), (4, 2, 8), (8, 2, 17), (12, 4, 5), (130, 1, 2)])
def test_decode_e4m3_row_counts(Hq, Hkv, nq):
    w = Batch([nq] * 4, [nq, 70, 300, 513], Hq=Hq, Hkv=Hkv, d=128, page=32, kind="e4m3", seed=Hq + nq)
    run_decode(w, nq, mask=MASK_CAUSAL, split=192)
    run_decode(w, nq, mask=MASK_CAUSAL, split=1 << 20)


@pytest.mark.parametrize("Hq,split", [(33, 64), (40, 192), (150, 64), (260, 320)])
def test_decode_e4m3_chunks_that_cut_a_tile(Hq, split):
    """More rows than the row kernel takes, in chunks that are no multiple of a key tile."""
    run_decode(Batch([1] * 7, LENS, Hq=Hq, Hkv=1, d=64, page=64, kind="e4m3", seed=34), 1,
               mask=MASK_CAUSAL, split=split)


def test_decode_e4m3_long_and_empty():
    w = Batch([1, 1], [20000, 4097], Hq=8, Hkv=1, d=128, page=64, kind="e4m3", seed=33)
    run_decode(w, 1, split=512)
    w = Batch([1, 1], [0, 0], Hq=4, Hkv=2, kind="e4m3", seed=34)
    run_decode(w, 1, max_seq_len=0)


def test_a_sequence_served_from_an_e4m3_cache():
    """Prompt in two chunks, then token by token, each step writing its tokens and attending
    to the cache: every output equals attention over the quantised keys and values, and the
    decode steps equal one-token chunks."""
    ea = _ea()
    d, Hq, Hkv, page, total = 64, 4, 2, 16, 90
    g = torch.Generator("cpu").manual_seed(35)
    q, k, v = (torch.randn(total, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pages = total // page + 1
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].cuda()
    kc, vc = (torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda") for _ in "kv")
    ex = torch.zeros(pages, Hkv, page, 2, dtype=torch.uint8, device="cuda")
    got_o, got_l, at = [], [], 0
    for n in [50, 30] + [1] * 10:
        sl = slice(at, at + n)
        at += n
        offs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lens = torch.tensor([at], dtype=torch.int32, device="cuda")
        ea.cache_write(k[sl].cuda(), v[sl].cuda(), kc, vc, table, offs, lens, kv_exp=ex)
        o, z = ea.prefill_paged(q[sl].cuda(), kc, vc, table, offs, lens, kv_exp=ex,
                                mask_kind=MASK_CAUSAL)
        if n == 1:
            od, zd = ea.decode_paged(q[sl].cuda()[None].transpose(1, 2).contiguous(), kc, vc, table,
                                     lens, kv_exp=ex)
            # the same row twice, each within its bound: with |O| <= A <= max |V| and V's own
            # rounding 2^-4, 2 (2^-8 + 2^-8 + 2^-11) (1 + 2^-4) max |V| < 5 * 2^-8 max |V|
            assert (od.reshape(o.shape).float() - o.float()).abs().max() <= 5 * 2.0 ** -8 * v.float().abs().max()
            assert (zd.reshape(z.shape) - z).abs().max() <= 4e-4
        got_o.append(o)
        got_l.append(z)
    kr, vr = ea.cache_read(kc, vc, table, torch.tensor([0, total], dtype=torch.int32, device="cuda"),
                           torch.tensor([total], dtype=torch.int32, device="cuda"), total, kv_exp=ex)
    kq, vq = P.decode(*P.encode(k.double().numpy())), P.decode(*P.encode(v.double().numpy()))
    assert np.array_equal(kr.double().cpu().numpy(), kq) and np.array_equal(vr.double().cpu().numpy(), vq)
    ref = P.chunk_forward(q, kc.cpu().numpy(), vc.cpu().numpy(), ex.cpu().numpy(), table.cpu().numpy(),
                          [0, total], [total], d ** -0.5, 1)
    check_attention(torch.cat(got_o), torch.cat(got_l), ref, "served")
    assert ea.device_status() == 0


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refusals():
    ea = _ea()
    w = Batch([3], [20], kind="e4m3", seed=40)
    c = w.cuda()
    pf = lambda **kw: ea.prefill_paged(*[{**c, **kw}[n] for n in (  # noqa: E731
        "q", "k_cache", "v_cache", "table", "offsets", "seq_lens")], kv_exp={**c, **kw}["kv_exp"])
    pf()
    for kw in (dict(kv_exp=None), dict(kv_exp=c["kv_exp"][:, :, :, :1].contiguous()),
               dict(k_cache=c["k_cache"].float()), dict(v_cache=c["v_cache"][1:]),
               dict(table=c["table"].long()), dict(offsets=c["offsets"][:1]),
               dict(seq_lens=c["seq_lens"].long()), dict(q=c["q"].float()), dict(q=c["q"].cpu()),
               dict(q=c["q"][..., :32]), dict(q=c["q"].transpose(1, 2).contiguous().transpose(1, 2)),
               dict(table=torch.cat([c["table"], c["table"]]))):
        with pytest.raises(ValueError):
            pf(**kw)
    wide = torch.zeros(3, w.Hq, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(ea.AttnError):
        pf(q=wide)   # a stride that is not a multiple of 8
    with pytest.raises(ValueError):
        ea.cache_write(c["k"], c["v"][:2], c["k_cache"], c["v_cache"], c["table"], c["offsets"],
                       c["seq_lens"], kv_exp=c["kv_exp"])
    with pytest.raises(ValueError):
        ea.decode_paged(c["q"][:1].transpose(0, 1)[None].contiguous(), c["k_cache"], c["v_cache"],
                        c["table"], c["seq_lens"])   # codes without exponents
