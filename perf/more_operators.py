"""Measurement cases of the operators around the paged cache that keep a serving loop on the
GPU: which sequence holds which page (fork, resize, compact), copies of pages between pools,
and the verification of drafted tokens, whose result says how far the cache is rolled back.

Conventions (include/attn.h has the full statement): caches are [pages, Hkv, page_size, d],
an e4m3 cache holds codes as uint8 and kv_exp uint8 [pages, Hkv, page_size, 2]. page_table is
int32 [B, max_pages], seq_lens int32 [B], and page_refs int32 [pages] counts the table entries
that hold a page: 0 is a free page. A negative entry holds no page (a sliding window has passed
it). All three are changed in place, so a pass here begins by putting them back.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    def pages(name, op, **kw):
        """B rows of len_min to len_max tokens, `beams` neighbours sharing their pages."""
        c = dict(name=name, op=op, kind="bf16", B=64, Hkv=8, d=128, page=64, len_min=512,
                 len_max=8192, beams=1, spare=500, grow_min=0, grow_max=1, empty=0.0, window=0)
        c.update(kw)
        return c

    def verify(name, **kw):
        c = dict(name=name, op="verify", kind="bf16", B=64, new_min=9, new_max=9, V=128000,
                 draft=True)
        c.update(kw)
        return c

    return [
        # beam search over few chats reorders its beams
        pages("fork_few", "fork", kind="bf16", B=8, Hkv=2, d=64, len_max=2000, beams=4, empty=0.2),
        # many long beams, small pages, some of them ending
        pages("fork_beams", "fork", B=512, Hkv=1, d=64, page=16, len_min=4000, len_max=16384,
              beams=8, empty=0.05),
        # a decode step of the repository's paged-decode benchmark: room for one token each
        pages("resize_step_bf16", "resize", grow_min=1),
        # the first step after a fork: every shared last page is copied before it is written
        pages("resize_after_fork_bf16", "resize", B=256, len_max=2048, beams=4, spare=1000,
              grow_min=1),
        # speculative steps over a sliding window: some rows roll back, some grow, some are new
        # prompts or have ended
        pages("resize_window_e4m3", "resize", kind="e4m3", B=160, Hkv=2, d=64, page=16,
              len_min=100, len_max=9000, spare=60000, grow_min=-8, grow_max=9, empty=0.25,
              window=4096),
        # a small pool is packed before a part of it is given up
        pages("compact_small_e4m3", "compact", kind="e4m3", B=12, Hkv=3, d=64, page=16,
              len_max=700, spare=300),
        # half of a serving pool is free, in no order
        pages("compact_half_bf16", "compact", B=64, spare=4400),
        # one request leaves for another pool
        pages("copy_few_e4m3", "copy", kind="e4m3", B=1, page=16, len_min=77, len_max=77, spare=40),
        # a batch is handed to another engine's pool
        pages("copy_batch_bf16", "copy", B=24, spare=500),
        # one sequence with four drafted tokens: latency
        verify("verify_one_fp32", kind="fp32", B=1, new_min=5, new_max=5, V=32000),
        # a batch of eight drafts each
        verify("verify_batch_bf16", B=128, V=128000),
        # drafts looked up in the prompt (no draft probabilities), ragged, an odd vocabulary
        verify("verify_lookup_fp16", kind="fp16", B=200, new_min=0, new_max=12, V=50257,
               draft=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "resize", "resize", "compact", "copy", "verify", "verify"])
    if op == "verify":
        c = dict(op=op, kind=rng.choice(["bf16", "fp16", "fp32"]), V=_log_int(rng, 300, 256000),
                 draft=rng.random() < 0.7)
        c["new_max"] = _log_int(rng, 1, 20)
        rows = 300_000_000 // c["V"]
        c["B"] = _log_int(rng, 1, max(1, min(600, rows // (2 * c["new_max"]))))
        c["new_min"] = rng.choice([0, 1, c["new_max"]])
        return c
    c = dict(op=op, kind=rng.choice(["bf16", "e4m3"]), Hkv=rng.choice([1, 2, 3, 4, 5, 8]),
             d=rng.choice([64, 128]), page=rng.choice([8, 16, 32, 64, 128, 192]),
             grow_min=0, grow_max=1, empty=rng.choice([0.0, 0.1, 0.5]), window=0)
    c["beams"] = rng.choice([1, 1, 2, 3, 5, 8]) if op in ("fork", "resize") else 1
    c["B"] = _log_int(rng, 1, 600)
    token = 2 * c["Hkv"] * c["d"] * (2 if c["kind"] == "bf16" else 1)
    most = min(400_000, 1_000_000_000 // token)               # cached tokens: at most 1 GB
    c["len_max"] = _log_int(rng, 1, max(2, min(30_000, most * c["beams"] // c["B"])))
    c["len_min"] = max(1, c["len_max"] // rng.choice([1, 3, 20]))
    c["spare"] = _log_int(rng, 1, max(2, most // c["page"]))
    if op == "resize":
        c["grow_max"] = _log_int(rng, 1, 2000)
        c["grow_min"] = rng.choice([0, 1, -c["grow_max"]])
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 2 * c["len_max"])])
        need = c["B"] * (c["grow_max"] // c["page"] + 2)
        need += int(c["empty"] * c["B"] + 1) * (c["len_max"] // c["page"] + 2)
        if need * c["page"] <= most and rng.random() < 0.9:   # else the pool may be too small
            c["spare"] += need
    return c


def _plan(case):
    """Lengths, sharing and requests of a case: a function of the case alone, so that work()
    and prepare() agree. Rows of a group of `beams` hold the same pages."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, ps = case["B"], case["page"]
    lens, group = [], []
    for b in range(B):
        if b % case["beams"] == 0:
            n = r.randint(case["len_min"], case["len_max"])
        lens.append(n)
        group.append(b // case["beams"])
    if case["op"] == "resize":                                # rows that wait for a prompt
        for g in range(group[-1] + 1):
            if r.random() < case["empty"] / 2:
                for b in range(B):
                    if group[b] == g:
                        lens[b] = 0
    need = [-(-lens[b] // ps) if b % case["beams"] == 0 else 0 for b in range(B)]
    parents, new = list(range(B)), list(lens)
    for b in range(B):
        first = group[b] * case["beams"]
        last = min(B, first + case["beams"]) - 1
        if case["op"] == "fork":
            parents[b] = -1 if r.random() < case["empty"] else r.randint(first, last)
        if case["op"] == "resize":
            if lens[b] == 0:
                new[b] = r.randint(case["len_min"], case["len_max"])
            elif r.random() < case["empty"] / 2:
                new[b] = 0                                    # the sequence has ended
            else:
                new[b] = max(1, lens[b] + r.randint(case["grow_min"], case["grow_max"]))
    most = -(-max(lens + new) // ps)
    return dict(lens=lens, need=need, parents=parents, new=new, max_pages=most + 2,
                pages=sum(need) + case["spare"])


def _drafts(case):
    r = random.Random("%d %d %d %d" % (case["B"], case["new_min"], case["new_max"], case["V"]))
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["B"])]
    if not sum(new):
        new[-1] = 1
    return new


def _page_bytes(case, tokens):
    return tokens * 2 * case["Hkv"] * (2 * case["d"] if case["kind"] == "bf16" else case["d"] + 1)


def work(case):
    if case["op"] == "verify":
        # the row of the first rejection, and the draft's beside it unless every token of the
        # sequence stays (about 3 of 4 drafted tokens do)
        size = 4 if case["kind"] == "fp32" else 2
        rows = sum(1 + (1 - 0.75 ** (n - 1) if case["draft"] else 0) for n in _drafts(case) if n)
        return {"bytes": rows * case["V"] * size + 16 * case["B"], "flops": 2 * rows * case["V"]}
    p, ps = _plan(case), case["page"]
    n = lambda t: -(-t // ps)  # noqa: E731
    held = sum(n(t) for t in p["lens"])
    if case["op"] == "fork":
        moved = sum(n(p["lens"][q]) for b, q in enumerate(p["parents"]) if q >= 0 and q != b)
        return {"bytes": 16 * moved + 12 * case["B"], "flops": held}
    if case["op"] == "resize":
        change = sum(abs(n(a) - n(b)) for a, b in zip(p["lens"], p["new"]))
        copied, at = 0, 0
        while at < case["B"]:                                 # one row of a group keeps its page
            rows = range(at, min(case["B"], at + case["beams"]))
            writes = [b for b in rows if p["new"][b] > p["lens"][b] and p["lens"][b] % ps]
            holds = sum(p["new"][b] * ps >= p["lens"][b] for b in rows)
            copied += max(0, len(writes) - (len(writes) >= holds)) * (p["lens"][at] % ps)
            at += case["beams"]
        return {"bytes": 4 * p["pages"] + 8 * change + 12 * case["B"] + 2 * _page_bytes(case, copied),
                "flops": p["pages"]}
    if case["op"] == "copy":
        return {"bytes": 2 * _page_bytes(case, held * ps) + 8 * held, "flops": held}
    used = sum(p["need"])                                     # pages behind the first `used`
    moved = int(used * (p["pages"] - used) / p["pages"])
    return {"bytes": 8 * p["pages"] + 8 * held + 2 * _page_bytes(case, moved * ps),
            "flops": p["pages"]}


# ------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _prepare_verify(case, g):
    """Probabilities of a target and of a draft model that agree on most of the mass, tokens
    drawn from the draft (or looked up: near the target's top), uniform random numbers."""
    new, V, dtype = _drafts(case), case["V"], _TYPES[case["kind"]]
    T = sum(new)
    offsets = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    target = torch.empty((T, V), dtype=dtype, device="cuda")
    draft = torch.empty((T, V), dtype=dtype, device="cuda") if case["draft"] else None
    tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
    step = max(1, 100_000_000 // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        logits = 2.5 * torch.randn((b - a, V), generator=g, device="cuda")
        p = torch.softmax(logits, -1)
        target[a:b] = p
        if draft is None:
            drawn = torch.topk(p, 3, dim=-1)[1][torch.arange(b - a), torch.randint(
                0, 3, (b - a,), generator=g, device="cuda")]
        else:
            q = torch.softmax(logits + 0.6 * torch.randn((b - a, V), generator=g, device="cuda"), -1)
            draft[a:b] = q
            drawn = torch.multinomial(q, 1, generator=g)[:, 0]
        end = min(T, b + 1)                                   # row t's draft is token t + 1
        tokens[a + 1:end] = drawn[:end - a - 1].to(torch.int32)
    accept = torch.rand(T, generator=g, device="cuda")
    if draft is None:                                         # a looked-up draft is often the text
        accept = accept * 0.002
    lens = torch.tensor([n + 100 for n in new], dtype=torch.int32, device="cuda")
    return dict(case=case, target=target, draft=draft, tokens=tokens, offsets=offsets, accept=accept,
                sample=torch.rand(len(new), generator=g, device="cuda"), lens=lens)


def _pool(case, num_pages, g):
    shape = (num_pages, case["Hkv"], case["page"], case["d"])
    out = []
    for _ in range(2):
        c = torch.empty(shape, dtype=torch.bfloat16 if case["kind"] == "bf16" else torch.uint8,
                        device="cuda")
        step = max(1, (1 << 27) // max(1, c[0].numel()))
        for p in range(0, num_pages, step):
            part = (min(num_pages, p + step) - p,) + shape[1:]
            if case["kind"] == "bf16":
                c[p:p + step] = torch.randn(part, generator=g, device="cuda")
            else:
                x = torch.randn(part, generator=g, device="cuda") * 100.0
                c[p:p + step] = x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        out.append(c)
    exp = None
    if case["kind"] == "e4m3":
        exp = torch.randint(118, 125, shape[:3] + (2,), generator=g, device="cuda",
                            dtype=torch.int32).to(torch.uint8)
    return out[0], out[1], exp


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(1000003 * seed + 29)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    plan = _plan(case)
    B, P, M = case["B"], plan["pages"], plan["max_pages"]
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((B, M), -1, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = plan["need"][b]
        if b % case["beams"] == 0:
            first, at = at, at + n
        held = perm[first:at]
        table[b, :len(held)] = held
        refs[held.long()] += 1
    # one buffer holds the integers that the operators change: table, lengths, counts
    saved = torch.cat([table.flatten(), torch.tensor(plan["lens"], dtype=torch.int32), refs]).cuda()
    live = saved.clone()
    cut = [live[:B * M].view(B, M), live[B * M:B * M + B], live[B * M + B:]]
    st = dict(case=case, saved=saved, live=live, table=cut[0], lens=cut[1], refs=cut[2])
    if case["op"] == "fork":
        st["parents"] = torch.tensor(plan["parents"], dtype=torch.int32, device="cuda")
        return st
    if case["op"] == "resize":
        st["new"] = torch.tensor(plan["new"], dtype=torch.int32, device="cuda")
    st["k"], st["v"], st["exp"] = _pool(case, P, g)
    if case["op"] == "copy":
        held = perm[:at]
        st["src"] = held.cuda()
        st["dst"] = torch.randperm(P, generator=g, device="cuda")[:at].to(torch.int32)
        st["k_to"], st["v_to"], st["exp_to"] = _pool(case, P, g)
    return st


# ------------------------------------------------------------------ plain forms
def _fork_plain(st):
    table, lens, refs, parents = st["table"], st["lens"], st["refs"], st["parents"].long()
    B, M = table.shape
    ps = st["case"]["page"]
    col, row = torch.arange(M, device="cuda")[None, :], torch.arange(B, device="cuda")
    n_old = (lens + ps - 1) // ps
    held = (col < n_old[:, None]) & (table >= 0)
    taken = torch.zeros(B, dtype=torch.int32, device="cuda")
    taken.index_add_(0, parents.clamp(min=0), (parents >= 0).int())
    refs.index_add_(0, table.clamp(min=0).flatten().long(),
                    torch.where(held, taken[:, None] - 1, 0).flatten().int())
    at = parents.clamp(min=0)
    new_lens = torch.where(parents >= 0, lens[at], 0)
    n_new = (new_lens + ps - 1) // ps
    moved = torch.where(col < n_new[:, None], table[at],
                        torch.where(col < n_old[:, None], -1, table))
    table.copy_(torch.where((parents == row)[:, None], table, moved))
    lens.copy_(new_lens)
    return table, lens, refs


def _resize_plain(st):
    case, table, lens, refs = st["case"], st["table"], st["lens"].long(), st["refs"]
    new = st["new"].long()
    ps, W = case["page"], case["window"]
    B, M = table.shape
    col, row = torch.arange(M, device="cuda")[None, :], torch.arange(B, device="cuda")
    n_old, n_new = (lens + ps - 1) // ps, (new + ps - 1) // ps
    # given back: pages behind the new length, and those that the window has passed, from its
    # edge down to the next entry that holds none
    gone = (col >= n_new[:, None]) & (col < n_old[:, None])
    if W:
        edge = ((torch.minimum(lens, new) - W + 1).clamp(min=0) // ps)[:, None]
        hole = torch.where((col < edge) & (table < 0), col, -1).amax(1, keepdim=True)
        gone = gone | ((col < edge) & (col > hole))
    drop = gone & (table >= 0)
    left = refs - torch.bincount(table[drop].long(), minlength=len(refs)).int()
    # the last page of a row that grows: copied first where others hold it
    at = (lens // ps).clamp(max=M - 1)
    writes = (new > lens) & (lens % ps > 0)
    page = table[row, at].long().clamp(min=0)
    many = torch.bincount(page[writes], minlength=len(refs))[page]
    lowest = torch.full((len(refs),), B, device="cuda").scatter_reduce_(
        0, page[writes], row[writes], "amin")[page]
    copy = writes & ((left[page] > many) | ((left[page] > 1) & (lowest != row)))
    fresh = (col >= n_old[:, None]) & (col < n_new[:, None])
    fresh = fresh | (copy[:, None] & (col == at[:, None]))
    need = fresh.sum()
    free = torch.nonzero(left == 0)[:, 0]
    missing = (need - len(free)).clamp(min=0).to(torch.int32).reshape(1)
    if int(missing):
        return table, st["lens"], refs, missing, st["k"], st["v"], st["exp"]
    free = free[:int(need)]
    left[free] = 1
    left -= torch.bincount(page[copy], minlength=len(refs)).int()
    table[gone] = -1
    table[fresh] = free.to(torch.int32)
    src, dst = page[copy], table[row, at][copy].long()
    used = (torch.arange(ps, device="cuda")[None, :] < (lens % ps)[copy][:, None])[:, None, :, None]
    for x in (st["k"], st["v"], st["exp"]):
        if x is not None:
            x[dst] = torch.where(used, x[src], x[dst])
    refs.copy_(left)
    st["lens"].copy_(new)
    return table, st["lens"], refs, missing, st["k"], st["v"], st["exp"]


def _compact_plain(st):
    table, lens, refs = st["table"], st["lens"], st["refs"]
    ps, P = st["case"]["page"], len(refs)
    used = refs != 0
    n = used.sum()
    index = torch.arange(P, device="cuda")
    src = torch.nonzero(used & (index >= n))[:, 0].flip(0)
    dst = torch.nonzero(~used & (index < n))[:, 0]
    for x in (st["k"], st["v"], st["exp"]):
        if x is not None:
            x[dst] = x[src]
    page_map = torch.where(used, index, -1)
    page_map[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    held = (torch.arange(table.shape[1], device="cuda")[None, :] < ((lens + ps - 1) // ps)[:, None])
    held = held & (table >= 0)
    table.copy_(torch.where(held, page_map[table.clamp(min=0).long()], table))
    return (table, lens, refs, n.to(torch.int32).reshape(1), page_map.to(torch.int32), st["k"],
            st["v"], st["exp"])


def _copy_plain(st):
    src, dst = st["src"].long(), st["dst"].long()
    for a, b in (("k", "k_to"), ("v", "v_to"), ("exp", "exp_to")):
        if st[a] is not None:
            st[b][dst] = st[a][src]
    return st["k_to"], st["v_to"], st["exp_to"]


def _verify_plain(st):
    offsets, tokens, V = st["offsets"].long(), st["tokens"].long(), st["target"].shape[1]
    B, T = len(offsets) - 1, len(tokens)
    new = offsets[1:] - offsets[:-1]
    some = new > 0
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new, output_size=T)
    i = torch.arange(T, device="cuda") - offsets[seq]
    last = i == new[seq] - 1
    token = tokens[(torch.arange(T, device="cuda") + 1).clamp(max=T - 1)].clamp(0, V - 1)[:, None]
    p = st["target"].gather(1, token)[:, 0].double()
    q = 1.0 if st["draft"] is None else st["draft"].gather(1, token)[:, 0].double()
    stays = (st["accept"].double() * q < p) & ~last
    stop = torch.where(stays, T, i)
    accepted = torch.full((B,), T, device="cuda").scatter_reduce_(0, seq, stop, "amin")
    accepted = torch.where(some, accepted, 0)
    row = (offsets[:-1] + accepted).clamp(max=T - 1)
    rejected = some & (accepted < new - 1)
    w = st["target"][row].double()
    if st["draft"] is None:
        left = w.scatter(1, token[row], 0.0)
    else:
        left = (w - st["draft"][row].double()).clamp(min=0)
    use = rejected & (left.sum(1) > 0)
    w = torch.where(use[:, None], left, w)
    total = w.cumsum(1)
    over = total > (st["sample"].double() * total[:, -1])[:, None]
    end = V - 1 - (w > 0).int().flip(1).argmax(1)             # the last token with any weight
    token = torch.where(over.any(1), over.int().argmax(1), end)
    token = torch.where(some, token, -1)
    kept = st["lens"] - torch.where(some, new - 1 - accepted, 0)
    return accepted.to(torch.int32), token.to(torch.int32), kept.to(torch.int32)


# ------------------------------------------------------------------ the framework's calls
def _run_own(st):
    import exact_io_aware_13_gb300 as ea
    op = st["case"]["op"]
    if op == "verify":
        return ea.verify_drafts(st["target"], st["tokens"], st["offsets"], st["accept"],
                                st["sample"], draft=st["draft"], seq_lens=st["lens"])
    if op == "copy":
        ea.cache_copy(st["k"], st["v"], st["k_to"], st["v_to"], st["src"], st["dst"],
                      kv_exp=st["exp"], kv_exp_to=st["exp_to"])
        return st["k_to"], st["v_to"], st["exp_to"]
    held = (st["table"], st["lens"], st["refs"])
    if op == "fork":
        ea.cache_fork(*held, st["parents"], page_size=st["case"]["page"])
        return held
    if op == "resize":
        missing = ea.cache_resize(st["k"], st["v"], *held, st["new"], kv_exp=st["exp"],
                                  window=st["case"]["window"])
        return held + (missing, st["k"], st["v"], st["exp"])
    return held + ea.cache_compact(st["k"], st["v"], *held, kv_exp=st["exp"]) + (
        st["k"], st["v"], st["exp"])


_PLAIN = {"fork": _fork_plain, "resize": _resize_plain, "compact": _compact_plain,
          "copy": _copy_plain, "verify": _verify_plain}


def run(state):
    op = state["case"]["op"]
    if op in ("fork", "resize", "compact"):
        state["live"].copy_(state["saved"])
    out = _run_own(state) if own else _PLAIN[op](state)
    if state["case"]["kind"] == "e4m3" and op != "fork":      # codes as the values they stand for
        out = tuple(x.view(torch.float8_e4m3fn) if x is not None and x.dim() == 4 and
                    x.shape[3] == state["case"]["d"] else x for x in out)
    return out


# ------------------------------------------------------------------ from the definitions
def _values(x):
    """Cache contents in 64 bits."""
    if x is None or x.dtype == torch.bfloat16:
        return x if x is None else x.to(torch.float64)
    c = torch.arange(256, device="cuda", dtype=torch.float64)
    s, e, m = c // 128, c // 8 % 16, c % 8
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10.0))
    v = torch.where(c % 128 == 127, math.nan, v) * (1 - 2 * s)
    return v[x.long()]


def _exact_verify(st):
    """One sequence after the other, one draft after the other."""
    offs, toks = st["offsets"].tolist(), st["tokens"].tolist()
    acc_u, smp_u, lens = st["accept"].tolist(), st["sample"].tolist(), st["lens"].tolist()
    accepted, nxt, kept = [], [], []
    for b in range(len(offs) - 1):
        a, n = 0, offs[b + 1] - offs[b]
        if n == 0:
            accepted.append(0), nxt.append(-1), kept.append(lens[b])
            continue
        w = None
        for t in range(offs[b], offs[b + 1] - 1):
            x, p = toks[t + 1], st["target"][t].double()
            q = torch.zeros_like(p) if st["draft"] is None else st["draft"][t].double()
            if st["draft"] is None:
                q[x] = 1.0
            if not acc_u[t] * float(q[x]) < float(p[x]):
                w = torch.relu(p - q)
                w = w if float(w.sum()) > 0 else p
                break
            a += 1
        w = st["target"][offs[b] + a].double() if w is None else w
        c = torch.cumsum(w, 0)
        x = int(torch.searchsorted(c, smp_u[b] * c[-1], right=True))
        accepted.append(a), kept.append(lens[b] - (n - 1 - a))
        nxt.append(min(x, int(torch.nonzero(w)[-1])))
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (accepted, nxt, kept))


def _exact_resize(case, st, table, lens, refs):
    """Row after row: releases first, then each row takes what it needs, on a list."""
    ps, W, new = case["page"], case["window"], st["new"].tolist()
    had = [x[:] for x in table], lens[:], refs[:]
    n = lambda t: -(-t // ps)  # noqa: E731
    for b, row in enumerate(table):
        for i in range(n(new[b]), n(lens[b])):
            if row[i] >= 0:
                refs[row[i]] -= 1
            row[i] = -1
        i = (min(lens[b], new[b]) - W + 1) // ps - 1 if W else -1
        while i >= 0 and row[i] >= 0:                         # page i ends before the window
            refs[row[i]] -= 1
            row[i] = -1
            i -= 1
    writers = {}
    for b, row in enumerate(table):
        if new[b] > lens[b] and lens[b] % ps:
            writers.setdefault(row[lens[b] // ps], []).append(b)
    copies = {b for e, rows in writers.items() for b in (rows if refs[e] > len(rows) else rows[1:])}
    free, taken, moves = [p for p, r in enumerate(refs) if r == 0], 0, []
    for b, row in enumerate(table):
        want = ([lens[b] // ps] if b in copies else []) + list(range(n(lens[b]), n(new[b])))
        for i in want:
            if taken < len(free):
                if i * ps < lens[b]:
                    moves.append((row[i], free[taken], lens[b] % ps))
                row[i] = free[taken]
            taken += 1
    if taken > len(free):
        return had + ([taken - len(free)], [])
    for p in free[:taken]:
        refs[p] = 1
    for src, _, _ in moves:
        refs[src] -= 1
    return table, new, refs, [0], moves


def exact(case, seed):
    st = prepare(case, seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "verify":
        return _exact_verify(st)
    if case["op"] == "copy":
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            for a, b in (("k", "k_to"), ("v", "v_to"), ("exp", "exp_to")):
                if st[a] is not None:
                    st[b][d].copy_(st[a][s])
        exps = None if st["exp"] is None else st["exp_to"].long()
        return _values(st["k_to"]), _values(st["v_to"]), exps
    table, lens, refs = st["table"].tolist(), st["lens"].tolist(), st["refs"].tolist()
    ps = case["page"]
    if case["op"] == "fork":
        par, old = st["parents"].tolist(), [r[:] for r in table]
        for b, row in enumerate(old):
            for e in row[:-(-lens[b] // ps)]:
                refs[e] -= 1
        new = [0 if p < 0 else lens[p] for p in par]
        for b, p in enumerate(par):
            for i in range(-(-max(lens[b], new[b]) // ps)):
                table[b][i] = old[p][i] if i * ps < new[b] else -1
                if i * ps < new[b]:
                    refs[table[b][i]] += 1
        return i32(table), i32(new), i32(refs)
    if case["op"] == "resize":
        table, lens, refs, missing, moves = _exact_resize(case, st, table, lens, refs)
        ints = i32(table), i32(lens), i32(refs), i32(missing)
    else:
        used = [p for p, r in enumerate(refs) if r]
        lo, hi, moves, where = 0, len(refs) - 1, [], {p: p for p in used}
        while True:                                           # two fingers meet
            while lo < len(refs) and refs[lo]:
                lo += 1
            while hi >= 0 and not refs[hi]:
                hi -= 1
            if lo >= hi:
                break
            moves.append((hi, lo, ps))
            where[hi], refs[lo], refs[hi] = lo, refs[hi], 0
        for b, row in enumerate(table):
            for i in range(-(-lens[b] // ps)):
                row[i] = where[row[i]]
        ints = (i32(table), i32(lens), i32(refs), i32([len(used)]),
                i32([where.get(p, -1) for p in range(len(refs))]))
    for src, dst, n in moves:
        for x in (st["k"], st["v"], st["exp"]):
            if x is not None:
                x[dst, :, :n] = x[src, :, :n]
    exps = None if st["exp"] is None else st["exp"].long()
    return ints + (_values(st["k"]), _values(st["v"]), exps)
