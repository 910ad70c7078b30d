"""The pool's operators together, as a serving loop makes them: beams that fork and go on,
drafted tokens that are scored, verified and rolled back, pages that a window has passed, and
pools that are compacted and handed over. Attention over what they leave has to be bit for bit
that over caches that were never shared, moved or rolled back."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _ea():
    import exact_io_aware_13_gb300 as ea
    return ea


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Cache:
    """A pool and its state; rows of tokens are written through resize and cache_write."""

    def __init__(self, B, M, pages, kind, Hkv=2, d=64, page=16, seed=0):
        self.ea, self.B, self.kind, self.Hkv, self.d, self.page = _ea(), B, kind, Hkv, d, page
        g = torch.Generator("cuda").manual_seed(seed)
        shape = (pages, Hkv, page, d)
        if kind == "bf16":                                   # free slots hold anything, NaN too
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            self.v, self.exp = self.k.clone(), None
        else:
            self.k, self.v = (torch.randint(0, 256, shape, generator=g, device="cuda").to(torch.uint8)
                              for _ in "kv")
            self.exp = torch.randint(0, 256, shape[:3] + (2,), generator=g, device="cuda").to(torch.uint8)
        self.table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")

    @property
    def state(self):
        return self.table, self.lens, self.refs

    def resize(self, new_lens, **kw):
        if not isinstance(new_lens, torch.Tensor):
            new_lens = i32(new_lens)
        missing = self.ea.cache_resize(self.k, self.v, *self.state, new_lens, kv_exp=self.exp, **kw)
        assert missing.tolist() == [0]

    def write(self, k, v, new, **kw):
        """new[b] tokens more for each row; k, v: the packed rows."""
        offs = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.resize(self.lens + i32(new), **kw)
        self.ea.cache_write(k, v, self.k, self.v, self.table, i32(offs), self.lens, kv_exp=self.exp)

    def decode(self, q, **kw):
        return self.ea.decode_paged(q, self.k, self.v, self.table, self.lens, kv_exp=self.exp, **kw)

    def tokens(self):
        """The cached rows of every sequence, read back."""
        lens = self.lens.tolist()
        offs = i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
        return self.ea.cache_read(self.k, self.v, self.table, offs, self.lens, sum(lens), kv_exp=self.exp)


def rows(n, seed, Hkv=2, d=64):
    g = torch.Generator("cuda").manual_seed(seed)
    return tuple(torch.randn(n, Hkv, d, generator=g, device="cuda").bfloat16() for _ in "kv")


def same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_beams(kind):
    """Six beams of two prompts: reordered, shared and written to for some steps."""
    c, plain = Cache(6, 20, 80, kind, seed=1), Cache(6, 20, 140, kind, seed=2)
    history = [[], [], [], [], [], []]                        # (step, packed row) of each token
    k, v = rows(77, 0)
    first = [29, 0, 0, 48, 0, 0]
    c.write(k, v, first)
    at = 0
    for b, n in enumerate(first):
        history[b] = [(k[t], v[t]) for t in range(at, at + n)]
        at += n
    rng = np.random.default_rng(3)
    parents = [0, 0, 0, 3, 3, 3]
    for step in range(9):
        c.ea.cache_fork(*c.state, i32(parents), page_size=c.page)
        history = [list(history[p]) for p in parents]
        k, v = rows(6, 10 + step)
        c.write(k, v, [1] * 6)
        for b in range(6):
            history[b].append((k[b], v[b]))
        parents = [int(rng.integers(0, 3)) + 3 * (b // 3) for b in range(6)]
    lens = [len(h) for h in history]
    assert c.lens.tolist() == lens
    plain.write(torch.stack([x[0] for h in history for x in h]),
                torch.stack([x[1] for h in history for x in h]), lens)
    same(c.tokens(), plain.tokens())
    q = torch.randn(6, 4, 1, 64, device="cuda").bfloat16()
    same(c.decode(q), plain.decode(q))
    # ended beams leave nothing behind
    c.ea.cache_fork(*c.state, i32([-1] * 6), page_size=c.page)
    assert int(c.refs.abs().sum()) == 0
    assert c.ea.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 40])
def test_speculative_steps(kind, window):
    """Drafted tokens are written, scored, verified and rolled back; the cache that is left, and
    attention over it, are those of the kept tokens alone."""
    ea, B, V = _ea(), 5, 300
    c, plain = Cache(B, 30, 60, kind, seed=4), Cache(B, 30, 160, kind, seed=5)
    mask = dict(mask_kind=ea.MASK_SLIDING_WINDOW, window=window) if window else dict(
        mask_kind=ea.MASK_CAUSAL)
    rng = np.random.default_rng(6)
    lens = [30, 61, 1, 16, 90]
    k, v = rows(sum(lens), 7)
    c.write(k, v, lens)
    plain.write(k, v, lens)
    g = torch.Generator("cuda").manual_seed(8)
    stayed = 0
    for step in range(8):
        new = [int(n) for n in rng.integers(0, 7, B)]
        if not sum(new):
            new[0] = 3
        offs, T = np.concatenate([[0], np.cumsum(new)]), sum(new)
        k, v = rows(T, 20 + step)
        c.write(k, v, new, window=window)
        q = torch.randn(T, 4, 64, generator=g, device="cuda").bfloat16()
        o, lse = ea.prefill_paged(q, c.k, c.v, c.table, i32(offs.tolist()), c.lens, kv_exp=c.exp, **mask)
        logits = torch.randn(T, V, generator=g, device="cuda")
        p, qd = torch.softmax(logits, -1), torch.softmax(logits + 0.5, -1).flip(0)
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda").int()
        u, u2 = torch.rand(T, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
        accepted, token, kept = ea.verify_drafts(p, tokens, i32(offs.tolist()), u, u2, draft=qd,
                                                 seq_lens=c.lens)
        before = c.lens.tolist()
        c.resize(kept, window=window)
        # the same step without what did not stay
        keep = [0 if n == 0 else 1 + a for n, a in zip(new, accepted.tolist())]
        stayed += sum(keep)
        assert c.lens.tolist() == [L - n + m for L, n, m in zip(before, new, keep)]
        idx = torch.tensor([int(offs[b]) + i for b in range(B) for i in range(keep[b])],
                           dtype=torch.int64, device="cuda")
        plain.write(k[idx], v[idx], keep)
        o2, lse2 = ea.prefill_paged(q[idx], plain.k, plain.v, plain.table,
                                    i32(np.concatenate([[0], np.cumsum(keep)]).tolist()), plain.lens,
                                    kv_exp=plain.exp, **mask)
        if max(new) == max(keep):                             # (else the tiles are others)
            assert torch.allclose(o[idx].float(), o2.float(), atol=2e-2)
    assert stayed > 0
    q = torch.randn(B, 4, 1, 64, device="cuda").bfloat16()
    same(c.decode(q, **mask), plain.decode(q, **mask))
    if window:
        assert int((c.refs > 0).sum()) < int((plain.refs > 0).sum())
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_compacted_and_handed_over(kind):
    ea = _ea()
    c = Cache(4, 20, 90, kind, seed=9)
    k, v = rows(500, 9)
    c.write(k, v, [200, 150, 100, 50])
    c.ea.cache_fork(*c.state, i32([0, -1, 2, 2]), page_size=16)
    q = torch.randn(4, 4, 1, 64, device="cuda").bfloat16()
    want, lens = c.decode(q), c.lens.tolist()
    read = c.tokens()
    used, page_map = ea.cache_compact(c.k, c.v, *c.state, kv_exp=c.exp)
    n = int(used)
    assert n == int((c.refs > 0).sum()) and int((c.refs[:n] == 0).sum()) == 0
    same(c.decode(q), want)
    same(c.tokens(), read)
    # the front of the pool alone, cut off
    cut = Cache(4, 20, n, kind, seed=10)
    pages = torch.arange(n, dtype=torch.int32, device="cuda")
    ea.cache_copy(c.k, c.v, cut.k, cut.v, pages, pages.flip(0).contiguous(), kv_exp=c.exp,
                  kv_exp_to=cut.exp)
    cut.table = torch.where(c.table >= 0, n - 1 - c.table, c.table)
    cut.lens = i32(lens)
    same(cut.decode(q), want)
    assert ea.device_status() == 0


def test_a_captured_step_replays():
    """Resize, write, scores, verification and roll-back as one graph, replayed on new inputs; a
    second graph of another pool runs beside it on its own workspaces."""
    ea, B, V, n = _ea(), 6, 500, 4
    offs, T = i32([n * b for b in range(B + 1)]), 6 * 4

    class Step:
        def __init__(self, seed):
            self.c = Cache(B, 40, 200, "bf16", seed=seed)
            k, v = rows(6 * 21, seed)
            self.c.write(k, v, [21] * 6)
            self.k, self.v = rows(T, seed + 1)
            self.p = torch.empty(T, V, device="cuda")
            self.tokens = torch.empty(T, dtype=torch.int32, device="cuda")
            self.u, self.u2 = torch.empty(T, device="cuda"), torch.empty(B, device="cuda")
            self.fill(seed)

        def fill(self, seed):
            g = torch.Generator("cuda").manual_seed(seed)
            self.p.copy_(torch.softmax(3 * torch.randn(T, V, generator=g, device="cuda"), -1))
            self.tokens.copy_(torch.cat([self.p.argmax(1)[-1:], self.p.argmax(1)[:-1]]).int())
            self.u.copy_(0.3 * torch.rand(T, generator=g, device="cuda"))
            self.u2.copy_(torch.rand(B, generator=g, device="cuda"))
            for x in (self.k, self.v):
                x.copy_(torch.randn(x.shape, generator=g, device="cuda"))

        def run(self):
            c = self.c
            missing = ea.cache_resize(c.k, c.v, *c.state, c.lens + n)
            ea.cache_write(self.k, self.v, c.k, c.v, c.table, offs, c.lens)
            a, t, kept = ea.verify_drafts(self.p, self.tokens, offs, self.u, self.u2, seq_lens=c.lens)
            ea.cache_resize(c.k, c.v, *c.state, kept)
            return missing, a, t

    steps, plain = [Step(50), Step(60)], [Step(50), Step(60)]
    graphs, outs = [], []
    for s in steps:
        saved = [x.clone() for x in (s.c.k, s.c.v, *s.c.state)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.synchronize()
        for x, y in zip((s.c.k, s.c.v, *s.c.state), saved):
            x.copy_(y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for i in (0, 1):
            steps[i].fill(100 * i + rep)
            plain[i].fill(100 * i + rep)
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            same(outs[i], plain[i].run())
            same(steps[i].c.state, plain[i].c.state)
            same(steps[i].c.tokens(), plain[i].c.tokens())
    assert ea.device_status() == 0


def test_calls_on_another_stream():
    """Allocating forms take no memory that the current stream still uses, and wait for nothing on
    it."""
    ea = _ea()
    c = Cache(3, 10, 40, "bf16", seed=1)
    k, v = rows(60, 1)
    c.write(k, v, [20, 30, 10])
    saved = [x.clone() for x in (c.k, c.v, *c.state)]
    p = torch.softmax(torch.randn(6, 700, device="cuda"), -1)
    tok, offs = torch.zeros(6, dtype=torch.int32, device="cuda"), i32([0, 2, 4, 6])
    u, u2 = torch.rand(6, device="cuda"), torch.rand(3, device="cuda")
    par, new = i32([1, 1, 0]), i32([31, 35, 0])
    src, dst = i32([c.table[0, 0]]), i32([39])

    def calls(stream):
        for x, y in zip((c.k, c.v, *c.state), saved):
            x.copy_(y)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)                         # some 10 ms on the current stream
        junk = [torch.full((m,), 255, dtype=torch.uint8, device="cuda") for m in (4, 512, 1024, 4096, 8192) * 3]
        del junk
        ea.cache_fork(*c.state, par, page_size=16, stream=stream)
        out = [ea.cache_resize(c.k, c.v, *c.state, new, stream=stream)]
        out += ea.cache_compact(c.k, c.v, *c.state, stream=stream)
        out += ea.verify_drafts(p, tok, offs, u, u2, seq_lens=c.lens, stream=stream)
        ea.cache_copy(c.k, c.v, c.k, c.v, src, dst, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        torch.cuda.synchronize()
        return [x.clone() for x in out + [c.k.view(torch.int16), c.v.view(torch.int16), *c.state]]

    want = calls(None)
    s = torch.cuda.Stream()
    for stream in (s, torch.cuda.ExternalStream(s.cuda_stream)):
        same(calls(stream), want)
    assert ea.device_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_callers_buffers_are_all_that_is_written(kind):
    """The forms with the caller's outputs and workspaces: the same results, and the bytes around
    every buffer keep what they held."""
    ea = _ea()

    class Guarded:
        def __init__(self, n):
            self.n, self.raw = n, torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
            self.view = self.raw[4096:4096 + n]

        def check(self):
            assert bool((self.raw[:4096] == 0xA5).all()) and bool((self.raw[4096 + self.n:] == 0xA5).all())

    def ints(n):
        g = Guarded(4 * n)
        return g, g.view.view(torch.int32)

    def pair():
        a = Cache(5, 9, 60, kind, seed=3)
        k, v = rows(150, 3)
        a.write(k, v, [50, 40, 30, 20, 10])
        a.ea.cache_fork(*a.state, i32([0, 0, 2, 3, -1]), page_size=16)
        return a
    a, b = pair(), pair()
    new = i32([53, 60, 0, 21, 144])
    want = ea.cache_resize(a.k, a.v, *a.state, new, kv_exp=a.exp)
    guards = []
    # the pool and its state inside guarded buffers
    for name in ("k", "v", "exp", "table", "lens", "refs"):
        x = getattr(b, name)
        if x is None:
            continue
        g = Guarded(x.nbytes)
        y = g.view.view(x.dtype).view(x.shape)
        y.copy_(x)
        setattr(b, name, y)
        guards.append(g)
    g, missing = ints(1)
    ws = Guarded(ea.resize_workspace_size(5, 9, 60))
    guards += [g, ws]
    ea.cache_resize_into(b.k, b.v, *b.state, new, missing, ws.view, kv_exp=b.exp)
    assert torch.equal(missing, want)
    parents = i32([4, 3, 2, 1, -1])
    ea.cache_fork(*a.state, parents, page_size=16)
    ws = Guarded(ea.fork_workspace_size(5, 9))
    guards.append(ws)
    ea.cache_fork(*b.state, parents, page_size=16, workspace=ws.view)
    want = ea.cache_compact(a.k, a.v, *a.state, kv_exp=a.exp)
    (g1, used), (g2, page_map) = ints(1), ints(60)
    ws = Guarded(ea.compact_workspace_size(60))
    guards += [g1, g2, ws]
    ea.cache_compact_into(b.k, b.v, *b.state, used, page_map, ws.view, kv_exp=b.exp)
    same((used, page_map), want)
    src, dst = torch.arange(40, dtype=torch.int32).cuda() % 20, torch.arange(40, dtype=torch.int32).cuda() + 20
    ea.cache_copy(a.k, a.v, a.k, a.v, src, dst, kv_exp=a.exp, kv_exp_to=a.exp)
    assert ea.device_status() == 0                            # (sources below 20, destinations from it on)
    ws = Guarded(ea.copy_workspace_size(60, 40))
    guards.append(ws)
    ea.cache_copy(b.k, b.v, b.k, b.v, src, dst, kv_exp=b.exp, kv_exp_to=b.exp, workspace=ws.view)
    assert ea.device_status() == 0
    same([x.view(torch.uint8) for x in (a.k, a.v, *a.state)], [x.view(torch.uint8) for x in (b.k, b.v, *b.state)])
    T, V = 9, 1001
    p = torch.softmax(torch.randn(T, V, device="cuda"), -1)
    tok, offs, lens = torch.ones(T, dtype=torch.int32, device="cuda"), i32([0, 3, 3, 9]), i32([9, 8, 7])
    u, u2 = torch.rand(T, device="cuda"), torch.rand(3, device="cuda")
    want = ea.verify_drafts(p, tok, offs, u, u2, seq_lens=lens)
    outs = [ints(3) for _ in range(3)]
    guards += [x[0] for x in outs]
    ea.verify_drafts_into(p, tok, offs, u, u2, outs[0][1], outs[1][1], seq_lens=lens, kept_lens=outs[2][1])
    same([x[1] for x in outs], want)
    torch.cuda.synchronize()
    for g in guards:
        g.check()
    assert ea.device_status() == 0
