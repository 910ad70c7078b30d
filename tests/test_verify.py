"""GPU parity of the verification of drafted tokens, against exact rational arithmetic (small
vocabularies) and float64 (large ones). The outputs are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

from oracle import pool_oracle as P

pytestmark = pytest.mark.gpu

BAD_INPUT = 8
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Drafts:
    """Ragged sequences of new[b] rows, probabilities of `kind`, on the CPU."""

    def __init__(self, new, V, kind="fp32", draft=True, seed=0, spare=0, noise=0.7):
        g = torch.Generator().manual_seed(seed)
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = self.T = int(self.offsets[-1]) + spare
        self.B, self.V, dtype = len(new), V, TYPES[kind]
        logits = 2 * torch.randn(T, V, generator=g)
        self.target = torch.softmax(logits, -1).to(dtype)
        q = torch.softmax(logits + noise * torch.randn(T, V, generator=g), -1)
        self.draft = q.to(dtype) if draft else None
        self.tokens = torch.zeros(T, dtype=torch.int32)
        if T > 1:
            drawn = torch.multinomial(q, 1, generator=g)[:-1, 0]
            self.tokens[1:] = (drawn if draft else self.target[:-1].float().argmax(1)).int()
        self.accept_u = torch.rand(T, generator=g)
        if not draft:
            self.accept_u *= 0.5
        self.sample_u = torch.rand(len(new), generator=g)
        self.lens = torch.randint(50, 100, (len(new),), generator=g, dtype=torch.int32)

    def want(self):
        f = lambda x: None if x is None else x.double().numpy()  # noqa: E731
        return P.verify(f(self.target), f(self.draft), self.tokens.numpy(), self.offsets,
                        self.accept_u.numpy(), self.sample_u.numpy())

    def run(self, target=None, draft=None, status=0, **kw):
        target = self.target.cuda() if target is None else target
        if draft is None and self.draft is not None:
            draft = self.draft.cuda()
        got = _ea().verify_drafts(target, self.tokens.cuda(), torch.from_numpy(self.offsets).cuda(),
                                  self.accept_u.cuda(), self.sample_u.cuda(), draft=draft,
                                  seq_lens=self.lens.cuda(), **kw)
        assert _ea().device_status() == status
        accepted, token, kept = (x.tolist() for x in got)
        new = np.diff(self.offsets)
        assert kept == [int(L) - max(0, int(n) - 1 - a)
                        for L, n, a in zip(self.lens, new, accepted)]
        return accepted, token

    def check(self, **kw):
        assert self.run(**kw) == tuple(self.want())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 64, 333, 1000])
def test_parity(kind, draft, V):
    Drafts([1, 0, 5, 2, 33, 0, 9, 70, 1], V, kind, draft, seed=V, spare=3).check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("V", [8191, 8193, 20_011])
def test_split_vocabularies(kind, V):
    """Several CTAs per sequence; exact sums over a vocabulary of their pieces."""
    Drafts([3, 1, 4], V, kind, True, seed=V).check()


def float64_want(w):
    """float64 over the GPU's copies; the margin tells that no rounding decides."""
    accepted, token = [], []
    for b in range(w.B):
        r0, r1 = int(w.offsets[b]), int(w.offsets[b + 1])
        t = r0
        while t < r1 - 1:
            x = int(w.tokens[t + 1])
            q = 1.0 if w.draft is None else float(w.draft[t, x])
            if not float(w.accept_u[t]) * q < float(w.target[t, x]):
                break
            t += 1
        p = w.target[t].double()
        if t < r1 - 1:
            if w.draft is None:
                p[int(w.tokens[t + 1])] = 0
            else:
                p = torch.relu(p - w.draft[t].double())
        c = torch.cumsum(p, 0)
        at = float(w.sample_u[b]) * float(c[-1])
        assert float((c - at).abs().min()) > 1e-11 * float(c[-1])
        accepted.append(t - r0)
        token.append(int(torch.searchsorted(c, at, right=True)))
    return accepted, token


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [32_000, 50_257, 128_000, 262_145])
def test_large_vocabularies(kind, draft, V):
    w = Drafts([5, 1, 3, 9], V, kind, draft, seed=V + draft)
    assert w.run() == float64_want(w)


def test_many_sequences():
    w = Drafts([int(n) for n in np.random.default_rng(0).integers(0, 6, 700)], 9001, "bf16", seed=5)
    got = w.run()
    live = np.diff(w.offsets) > 0
    assert [a for a, x in zip(got[0], live) if not x] == [0] * int((~live).sum())
    assert [a for a, x in zip(got[1], live) if not x] == [-1] * int((~live).sum())
    keep = np.flatnonzero(live)[::7]
    w2 = float64_want_of(w, keep)
    assert [(got[0][b], got[1][b]) for b in keep] == w2


@pytest.mark.parametrize("kind,draft", [("bf16", True), ("fp32", False)])
def test_long_pieces(kind, draft):
    """So many sequences that one CTA has a whole vocabulary, in several pieces per warp."""
    w = Drafts([1] * 300 + [3, 2, 1, 4], 70_003, kind, draft, seed=6)
    got = w.run()
    keep = list(range(0, 300, 43)) + [300, 301, 302, 303]
    assert [(got[0][b], got[1][b]) for b in keep] == float64_want_of(w, keep)


def float64_want_of(w, which):
    import copy
    out = []
    for b in which:
        one = copy.copy(w)
        r0, r1 = int(w.offsets[b]), int(w.offsets[b + 1])
        one.B, one.offsets = 1, np.array([0, r1 - r0], dtype=np.int32)
        one.target, one.draft = w.target[r0:r1], None if w.draft is None else w.draft[r0:r1]
        one.tokens, one.accept_u = w.tokens[r0:r1], w.accept_u[r0:r1]
        one.sample_u = w.sample_u[b:b + 1]
        a, t = float64_want(one)
        out.append((a[0], t[0]))
    return out


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("p_off,q_off,pad", [(0, 0, 3), (1, 1, 0), (3, 1, 5), (0, 7, 1), (2, 0, 13)])
def test_strides_and_alignments(kind, p_off, q_off, pad):
    """Rows that start anywhere, p and q at different distances from a 16-byte boundary."""
    w = Drafts([4, 1, 6], 513, kind, True, seed=p_off + 10 * pad)
    def view(x, off):
        big = torch.full((w.T, w.V + off + pad), float("nan"), dtype=x.dtype, device="cuda")
        big[:, off:off + w.V] = x.cuda()
        return big[:, off:off + w.V]
    w.check(target=view(w.target, p_off), draft=view(w.draft, q_off))


def test_one_row_view_of_a_transposed_batch():
    """A broadcast target (row stride 0) is read as the same row for all."""
    w = Drafts([3, 2], 100, "fp32", seed=3)
    w.target = w.target[:1].expand(w.T, w.V)
    w.check(target=w.target[:1].cuda().expand(w.T, w.V))


@pytest.mark.parametrize("kind", list(TYPES))
def test_random_numbers_at_the_ends(kind):
    for u in (0.0, 2.0 ** -40, 1 - 2.0 ** -24):
        w = Drafts([1, 4, 3], 300, kind, seed=8)
        w.sample_u[:] = u
        w.check()
        w.accept_u[:] = u
        w.check()
    w.target[:, 100:] = 0                                     # the last tokens have no weight
    w.accept_u[:] = 0.999
    w.sample_u[:] = 1 - 2.0 ** -24
    w.check()
    assert max(w.run()[1]) < 100


def test_what_is_not_read():
    """The rows of draft, random numbers and tokens that the rule does not name may hold anything."""
    w = Drafts([4, 1, 0, 3], 300, "fp32", seed=12, spare=2)
    want = w.run()
    last = [int(o) - 1 for o in w.offsets[1:]] + [w.T - 2, w.T - 1]
    w.draft[last] = float("nan")
    w.accept_u[last] = float("nan")
    w.target[w.T - 2:] = float("nan")
    w.tokens[[int(o) for o in w.offsets[:-1]]] = -5
    w.tokens[w.T - 2:] = 10 ** 9
    w.sample_u[2] = float("nan")                              # of the sequence without rows
    assert w.run() == want


def test_more_sequences_than_a_grid_holds_at_once():
    w = Drafts([1, 2, 0, 3] * 5000, 37, "fp16", seed=13)
    got = w.run()
    part = Drafts([1, 2, 0, 3] * 5000, 37, "fp16", seed=13)
    part.B, T = 400, int(part.offsets[400])
    part.offsets, part.lens, part.sample_u = part.offsets[:401], part.lens[:400], part.sample_u[:400]
    part.T, part.target, part.draft = T, part.target[:T], part.draft[:T]
    part.tokens, part.accept_u = part.tokens[:T], part.accept_u[:T]
    want = part.want()
    assert (got[0][:400], got[1][:400]) == tuple(want)
    assert all(0 <= t < 37 for t, n in zip(got[1], np.diff(w.offsets)) if n)


def test_the_binding_refuses():
    ea = _ea()
    w = Drafts([3, 2], 50, "fp32", seed=1)
    good = dict(target=w.target.cuda(), tokens=w.tokens.cuda(), offsets=i32(w.offsets), accept_u=w.accept_u.cuda(),
                sample_u=w.sample_u.cuda(), draft=w.draft.cuda(), seq_lens=w.lens.cuda())
    for bad in (dict(target=good["target"].double()), dict(target=good["target"].t().contiguous().t()),
                dict(draft=good["draft"].half()), dict(draft=good["draft"][:4]), dict(draft=good["draft"][:, :49]),
                dict(tokens=good["tokens"].long()), dict(tokens=good["tokens"][:4]), dict(offsets=i32([])),
                dict(accept_u=good["accept_u"].double()), dict(accept_u=good["accept_u"][:4]),
                dict(sample_u=good["sample_u"][:1]), dict(seq_lens=i32([1])), dict(target=w.target),
                dict(target=good["target"][0])):
        with pytest.raises(ValueError):
            ea.verify_drafts(**{**good, **bad})
    out = i32([0, 0])
    kw = {k: v for k, v in good.items() if k != "seq_lens"}
    with pytest.raises(ValueError, match="needs seq_lens"):
        ea.verify_drafts_into(accepted=out, next_tokens=out.clone(), kept_lens=out.clone(), **kw)
    ea.verify_drafts(**good)
    assert ea.device_status() == 0


def test_equal_distributions():
    """p = q: every draft stays unless u = 1 - ... rounds; a forced rejection draws from p."""
    w = Drafts([5, 2], 700, "fp32", seed=2)
    w.draft = w.target.clone()
    w.check()
    assert w.run()[0] == [4, 1]
    w.accept_u[:] = 1.0                                       # u q < p fails: no residual is left
    w.check()
    assert w.run()[0] == [0, 0]
    for V in (40_000, 200_001):
        forced_rejection(V)


def forced_rejection(V):
    big = Drafts([2, 3], V, "bf16", seed=2)
    big.draft, big.accept_u[:] = big.target.clone(), 1.0
    accepted, token = big.run()
    assert accepted == [0, 0]
    for b, t in enumerate((0, 2)):
        c = torch.cumsum(big.target[t].double(), 0)
        assert token[b] == int(torch.searchsorted(c, float(big.sample_u[b]) * float(c[-1]), right=True))


def test_weights_that_are_no_numbers():
    w = Drafts([1, 3, 1, 4], 200, "fp32", seed=4)
    inf, nan = float("inf"), float("nan")
    w.target[:, 3], w.target[:, 50], w.target[:, 90], w.target[:, 199] = nan, inf, -inf, -1.0
    w.draft[:, 60], w.draft[:, 61] = nan, inf
    w.tokens[:] = 7
    w.check()
    w.target[0] = nan                                         # a row without any weight
    w.target[int(w.offsets[2])] = 0.0
    got = w.run(status=BAD_INPUT)
    assert got[1][0] == -1 and got[1][2] == -1
    assert got == tuple(w.want())


def test_drafts_whose_probabilities_are_no_numbers():
    """Neither an infinite nor a NaN probability lets a draft stay, whatever its random number."""
    inf, nan = float("inf"), float("nan")
    for u in (0.0, 0.5):
        for p, q in ((inf, 0.5), (nan, 0.5), (-inf, 0.5), (-0.25, -0.5), (0.0, 0.0), (0.5, nan), (0.5, inf),
                     (0.5, -inf), (0.25, 0.0), (2.0 ** -149, 2.0 ** -149), (3e38, 3e38)):
            w = Drafts([3, 2], 40, "fp32", seed=4)
            w.tokens[:] = 9
            w.target[:, 9], w.draft[:, 9], w.accept_u[:] = p, q, u
            w.check()


def test_tiny_weights_count():
    """Probabilities in fp32's subnormal range, residuals that cancel to their last bits."""
    w = Drafts([1, 2, 2], 400, "fp32", seed=6)
    w.target[0] = 0
    w.target[0, [5, 77, 300]] = torch.tensor([2.0 ** -149, 2.0 ** -148, 2.0 ** -149])
    w.draft = w.target.clone()
    for t in (1, 3):
        x = torch.arange(0, 400, 3)
        w.draft[t, x] = torch.nextafter(w.draft[t, x], torch.tensor(0.0))
    w.accept_u[:] = 1.0
    for u in (0.1, 0.3, 0.6, 0.9):
        w.sample_u[:] = u
        w.check()


def test_bad_device_inputs_are_reported():
    w = Drafts([3, 2], 50, "fp32", seed=1)
    w.tokens[1] = 50                                          # outside the vocabulary: rejected
    got = w.run(status=BAD_INPUT)
    assert got[0][0] == 0 and 0 <= got[1][0] < 50
    w = Drafts([3, 2], 50, "fp32", seed=1)
    for offsets in ([0, 4, 3], [0, -1, 5], [0, 3, 6], [1, 3, 5]):
        w.offsets = np.array(offsets, dtype=np.int32)
        ea = _ea()
        ea.verify_drafts(w.target.cuda(), w.tokens.cuda(), i32(offsets), w.accept_u.cuda(),
                         w.sample_u.cuda(), draft=w.draft.cuda())
        assert ea.device_status() == BAD_INPUT, offsets


def test_empty_calls():
    ea = _ea()
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    a, t = ea.verify_drafts(f(0, 10), i32([]), i32([0]), f(0), f(0))
    assert a.shape == t.shape == (0,)
    a, t = ea.verify_drafts(f(0, 10), i32([]), i32([0, 0, 0]), f(0), f(2))
    assert a.tolist() == [0, 0] and t.tolist() == [-1, -1]
    assert ea.device_status() == 0
    a, t = ea.verify_drafts(f(1, 0), i32([0]), i32([0, 1]), f(1), f(1))  # no vocabulary
    assert a.tolist() == [0] and t.tolist() == [-1]
    assert ea.device_status() == BAD_INPUT
