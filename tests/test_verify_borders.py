"""Verification of drafted tokens where u * total lies close to a border between two tokens: totals
and random numbers in fp32's subnormal range, and borders inside long vocabularies. The expected
tokens come from whole-number arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.test_verify import TYPES, Drafts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


# ------------------------------------------------------------------ totals near zero
@pytest.mark.parametrize("u", [0.1, 0.2, 0.3, 0.4, 0.5, 0.6, 0.7, 0.8, 0.9, 1 - 2.0 ** -24])
def test_totals_of_a_few_subnormal_steps(u):
    """The product of u and the total is no multiple of fp32's smallest step."""
    w = Drafts([1, 2, 2], 400, "fp32", seed=6)
    w.target[0] = 0
    w.target[0, [5, 77, 300]] = torch.tensor([2.0 ** -149, 2.0 ** -148, 2.0 ** -149])
    w.draft = w.target.clone()
    for t in (1, 3):                                          # residuals of a last bit here and there
        x = torch.arange(0, 400, 3)
        w.draft[t, x] = torch.nextafter(w.draft[t, x], torch.tensor(0.0))
    w.accept_u[:] = 1.0
    w.sample_u[:] = u
    w.check()


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("exponent", [-149, -148, -140, -126, -120, -100, -80, -76, -60, -50, 0, 100])
def test_totals_of_any_size(exponent, draft):
    """Weights of one to nine steps of 2^exponent in rows of zeros, and residuals of such weights."""
    for seed in range(12):
        w = Drafts([1, 2, 1, 3], 90, "fp32", draft=draft, seed=seed)
        rng = np.random.default_rng(100 + seed)
        for t in range(w.T):
            steps = rng.integers(1, 10, w.V) * (rng.random(w.V) < 0.15)
            w.target[t] = torch.from_numpy(steps.astype(np.float64) * 2.0 ** exponent).float()
            if draft:
                w.draft[t] = w.target[t] * torch.from_numpy(rng.integers(0, 3, w.V)).float()
            w.target[t, 50] = 2.0 ** exponent
        w.accept_u[:] = 1.0                                   # nothing stays that is not certain
        w.check()


def test_random_numbers_near_zero():
    """u * total below fp32's smallest step, in front of weights of one such step."""
    for u in (2.0 ** -149, 3 * 2.0 ** -149, 2.0 ** -126, 0.75 * 2.0 ** -99, 1.25 * 2.0 ** -99, 2.0 ** -99,
              1.5 * 2.0 ** -99, 2.0 ** -60, 2.0 ** -30):
        for big in (2.0 ** -100, 2.0 ** -50, 1.0, 2.0 ** 100):
            w = Drafts([1, 1], 300, "fp32", seed=1)
            w.target[:] = 0
            w.target[:, [4, 5, 6]] = 2.0 ** -149
            w.target[:, 200] = big
            w.target[1, 7] = 2.0 ** -130
            w.sample_u[:] = u
            w.check()


# ------------------------------------------------------------------ borders in long vocabularies
# A lane sums n of a row's weights in each half of a pair of fp32 numbers (hi, lo). Every weight
# brings lo a two-sum error and a residual's rounding error, each at most e = 2^-24 of the lane's
# sum S, so |lo| <= (n + 1) e S, and its two additions round by e |lo| each: 2 n (n + 1) e^2 S in
# all. Joining pairs (five steps over the lanes, at most 8 + 5 over the pieces, 16 + 5 + 5 inside
# the piece that holds the token) rounds lo by at most 3 e^2 S each, the threshold by as much. Here
# pieces have at most 1024 elements (one sequence has at least 64 warps from 32768 tokens on, 128000
# tokens have 128): n is 16, and 544 + 3 * 45 = 679 e^2 of the total is 2^-38.6. Borders lie 2^-37 of
# the total away.
DISTANCE = Fraction(1, 1 << 37)
UNIT = 149 + 24


def whole(x):
    """fp32 values as whole numbers of 2^-UNIT, so that sums and products of them are exact."""
    m, e = np.frexp(x.double().numpy())
    return [int(a) << int(b) for a, b in zip((m * 2.0 ** 24).astype(np.int64), e - 24 + UNIT)]


def floor_to(value, dtype):
    """The largest number of the type that is not above a positive fraction (0 if there is none)."""
    x = torch.tensor(float(value), dtype=torch.float64).to(dtype)
    if Fraction(float(x)) > value:
        x = torch.nextafter(x.float(), torch.tensor(0.0)) if dtype == torch.float32 else (
            x.view(torch.int16) - 1).view(dtype)
    return x


def border_row(kind, V, seed, side, draft):
    """p (and q) of a row and u such that a running sum passes u * total by `side` * DISTANCE."""
    g = torch.Generator().manual_seed(seed)
    dtype = TYPES[kind]
    scale = 2.0 ** 9 if kind == "fp16" else 2.0 ** -15        # (rows need not sum to one)
    p = (scale * torch.rand(V, generator=g)).to(dtype)
    q = (p.float() * (0.4 + torch.rand(V, generator=g))).to(dtype) if draft else None
    tune = list(range(8))
    p[tune] = 0
    if draft:
        q[tune] = 0
    u = float(torch.tensor(0.05 + 0.9 * float(torch.rand((), generator=g, dtype=torch.float64))).float())
    w = whole(p)
    if draft:
        w = [max(0, a - b) for a, b in zip(w, whole(q))]
    run = np.cumsum(np.array(w, dtype=object))
    U = Fraction(u)
    at = int(np.searchsorted(run, U * int(run[-1]), side="right"))  # the border is in front of `at`
    assert 100 < at < V - 100
    # weights a_k in front raise the running sum by a and the threshold by u a
    total = int(run[-1])
    want = (U * total - int(run[at - 1]) + side * DISTANCE * total) / (1 - U)
    assert want > 0
    for x in tune:
        a = floor_to(want / (1 << UNIT), dtype)
        p[x] = a
        want -= Fraction(float(a)) * (1 << UNIT)
    w = whole(p)
    if draft:
        w = [max(0, a - b) for a, b in zip(w, whole(q))]
    run = np.cumsum(np.array(w, dtype=object))
    gap = (int(run[at - 1]) - U * int(run[-1])) / int(run[-1])
    assert abs(gap - side * DISTANCE) < DISTANCE / 8
    return p, q, u, int(np.searchsorted(run, U * int(run[-1]), side="right"))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [20_011, 50_257, 128_000])
def test_borders_of_long_vocabularies(kind, draft, V):
    """The border just passed, and just not: two neighbouring tokens, each the right one once."""
    for seed in range(3):
        tokens = []
        for side in (1, -1):
            p, q, u, want = border_row(kind, V, 1000 * seed + V, side, draft)
            w = Drafts([2 if draft else 1], V, kind, draft, seed=0)
            w.target[0], w.sample_u[:], w.accept_u[:] = p, u, 1.0
            if draft:                                         # a draft that does not stay
                w.draft[0] = q
                x = int(torch.nonzero(q.float() > p.float())[0])
                w.tokens[1] = x
            got = w.run()
            assert got == ([0], [want]), (seed, side)
            tokens.append(want)
        assert tokens[0] < tokens[1]


@pytest.mark.parametrize("V", [4096, 65_536, 131_072])
def test_borders_that_are_met(V):
    """Equal weights of 2^-k: u * total is a running sum itself, which does not exceed it."""
    rng = np.random.default_rng(V)
    for x in [0, 1, V // 2, V - 1, *rng.integers(0, V, 5).tolist()]:
        w = Drafts([1], V, "bf16", draft=False)
        w.target[:] = 1.0 / V
        for u, want in ((x / V, x), (np.nextafter(np.float32(x / V), np.float32(1)), x),
                        (np.nextafter(np.float32(x / V), np.float32(0)), max(x - 1, 0))):
            w.sample_u[:] = float(u)
            assert w.run() == ([0], [want]), (x, u)
