"""Operators of a serving step beside the Q2_0 products, as cases to time and compare.

  route    expert choice from softmax or sigmoid scores with a bias for balance, inside the best groups
  verify   drafted tokens against the target's probabilities, and the token that follows the accepted ones
  copy     pages of a paged cache to other places, and a whole pool into another without its free pages
  steps    what a scheduler does to the page tables between two model steps: sequences shrink and grow (a
           rejected draft's pages go back, an ended sequence's, a new prompt's are taken), and fork

`run` computes an operator in plain torch operations (32 bits; 64 where scores or sums decide between two
choices), or (own = True) through the package's entry points; `exact` computes it in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # the router of one decoded token: latency counts
        dict(name="route_1", op="route", tokens=1, experts=128, used=8, groups=8, groups_used=4, top=2, score="sigmoid", x="f32",
             bias=True, normalise=True),
        # a prompt batch over many experts in groups
        dict(name="route_4096", op="route", tokens=4096, experts=256, used=8, groups=8, groups_used=4, top=2, score="sigmoid",
             x="f32", bias=True, normalise=True),
        # softmax scores, groups of an odd size, the group's best expert decides, weights as they are
        dict(name="route_odd_777", op="route", tokens=777, experts=60, used=6, groups=5, groups_used=3, top=1, score="softmax",
             x="bf16", bias=False, normalise=False),
        # one chat with four drafted tokens
        dict(name="verify_chat_1", op="verify", seqs=1, drafts=4, vocab=151936, form="logits", draft=True, temp="one", x="f32"),
        # an ordinary batch whose drafts come from its own text (no draft model), an odd vocabulary of 16-bit logits
        dict(name="verify_lookup_16", op="verify", seqs=16, drafts=5, vocab=50001, form="logits", draft=False, temp="mixed", x="bf16"),
        # both models' probabilities are there already
        dict(name="verify_probs_32", op="verify", seqs=32, drafts=3, vocab=32003, form="probs", draft=True, temp="one", x="f32"),
        # a large batch, some of its requests greedy
        dict(name="verify_batch_64", op="verify", seqs=64, drafts=4, vocab=151936, form="logits", draft=True, temp="mixed", x="f32"),
        # the pages of sequences that are swapped out, into a pool of another layout
        dict(name="copy_swap_1024", op="copy", pages=1800, n=1024, page=64, n_kv=8, dim=128, cache="bf16", layout="tokens"),
        # a pool of which a third is in use moves into a smaller one
        dict(name="compact_6000", op="compact", pages=6000, to_pages=2600, seqs=24, shared=200, used=2100, page=16, n_kv=8, dim=128,
             cache="bf16"),
        # between two steps of a batch that drafts 8 tokens: the rejected ones go, rows for the next are taken
        dict(name="steps_drafts_64", op="steps", kind="drafts", seqs=64, lo=900, hi=12000, drafts=8, page=16, n_kv=4, dim=128,
             cache="bf16"),
        # beams: in each group of four two end and the other two fork, then all go on, in pages of their own
        dict(name="steps_beams_32", op="steps", kind="beams", seqs=32, lo=700, hi=3500, drafts=0, page=16, n_kv=8, dim=128,
             cache="f16"),
        # half of a large batch ends, and new prompts take their places
        dict(name="steps_turnover_256", op="steps", kind="turnover", seqs=256, lo=1000, hi=16000, drafts=0, page=16, n_kv=1, dim=64,
             cache="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "verify", "verify", "verify", "copy", "compact", "steps", "steps"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
        size = _log(rng, 2, 512 // groups)
        picked = rng.randint(1, groups)
        return dict(op=op, tokens=_log(rng, 1, 4000) | 1, experts=groups * size, used=rng.randint(1, min(8, picked * size)),
                    groups=groups, groups_used=picked, top=rng.choice([1, 2]), score=rng.choice(["softmax", "sigmoid"]),
                    x=rng.choice(["f32", "bf16", "f16"]), bias=rng.choice([True, True, False]), normalise=rng.choice([True, False]))
    if op == "verify":
        vocab, drafts = _log(rng, 500, 151936), rng.choice([0, 1, 2, 3, 4, 5, 7, 15])
        most = max(1, min(64, 64 * 9 * 151936 // ((2 * drafts + 1) * vocab)))      # within the largest listed case
        form = rng.choice(["logits", "logits", "probs"])
        return dict(op=op, seqs=_log(rng, 1, most), drafts=drafts, vocab=vocab, form=form, draft=drafts > 0 and rng.random() < 0.7,
                    temp="one" if form == "probs" else rng.choice(["one", "mixed"]),
                    x="f32" if form == "probs" else rng.choice(["f32", "f32", "bf16", "f16"]))
    page, n_kv, dim = rng.choice([16, 16, 20, 64]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    cache = rng.choice(["bf16", "f16"])
    rows = 1800 * 64 * 8 * 128 // (page * n_kv * dim)                              # pages of the largest listed pool
    if op == "copy":
        pages = _log(rng, 8, min(6000, rows))
        return dict(op=op, pages=pages, n=_log(rng, 1, max(1, pages // 2)), page=page, n_kv=n_kv, dim=dim, cache=cache,
                    layout=rng.choice(["heads", "tokens"]))
    if op == "compact":
        pages = _log(rng, 100, min(6000, rows))
        used = max(20, int(pages * rng.uniform(0.2, 0.35)))
        return dict(op=op, pages=pages, to_pages=used + rng.randint(0, pages // 4), seqs=rng.randint(1, 16), shared=rng.randint(0, 8),
                    used=used, page=page, n_kv=n_kv, dim=dim, cache=cache)
    kind = rng.choice(["drafts", "beams", "turnover"])
    seqs = 4 * _log(rng, 1, 32)
    hi = _log(rng, 100, max(100, min(12000, rows * page // (2 * seqs))))
    return dict(op=op, kind=kind, seqs=seqs, lo=max(20, hi // rng.choice([1, 3, 10])), hi=hi, drafts=rng.randint(1, 15), page=page,
                n_kv=n_kv, dim=dim, cache=cache)


# ----------------------------------------------------------------------- sizes of a case

def _size(name):
    return {"f32": 4, "f16": 2, "bf16": 2}[name]


def _lens(c):
    """Lengths of the sequences, spread evenly over [lo, hi]; not a whole number of pages, so that beams fork inside one."""
    n = c["seqs"]
    got = [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) for i in range(n)]
    return [v + 1 if v % c["page"] == 0 else v for v in got]


def _page_bytes(c):
    return 2 * c["page"] * c["n_kv"] * c["dim"] * 2              # keys and values


def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": c["tokens"] * (c["experts"] * _size(c["x"]) + c["used"] * 8) + (4 * c["experts"] if c["bias"] else 0),
                "flops": c["tokens"] * c["experts"] * 6}
    if c["op"] == "verify":
        if c["form"] == "probs":                                 # the row of the first rejection alone, and its draft's
            rows = c["seqs"] * (2 if c["draft"] else 1)
        else:
            rows = c["seqs"] * (c["drafts"] + 1 + (c["drafts"] if c["draft"] else 0))
        return {"bytes": rows * c["vocab"] * _size(c["x"]) + c["seqs"] * (c["drafts"] + 1) * 12, "flops": 4 * rows * c["vocab"]}
    if c["op"] == "copy":
        return {"bytes": c["n"] * (2 * _page_bytes(c) + 8), "flops": 0}
    if c["op"] == "compact":
        return {"bytes": c["used"] * (2 * _page_bytes(c) + 4 + 4 + 8), "flops": 0}
    # entries of the tables that change (old, new, and the page's count twice), and the lengths
    n, page = c["seqs"], c["page"]
    pages = [-(-v // page) for v in _lens(c)]
    if c["kind"] == "drafts":
        changed, rows = n * c["drafts"] / page, 0
    elif c["kind"] == "beams":                                   # half the sequences go and come again
        changed, rows = sum(pages), sum(v % page for v in _lens(c)) / 2
    else:
        changed, rows = sum(pages), 0                            # half of them, twice
    return {"bytes": changed * 16 + n * 16 + rows * 2 * _page_bytes(c) / page, "flops": 0}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _pools(g, c, pages, layout="heads"):
    """Two pools (pages, n_kv, page, dim); layout "tokens": the heads of a token next to each other in memory."""
    dt = DTYPES[c["cache"]]
    if layout == "heads":
        return [_randn(g, pages, c["n_kv"], c["page"], c["dim"]).to(dt) for _ in range(2)]
    return [_randn(g, pages, c["page"], c["n_kv"], c["dim"]).to(dt).transpose(1, 2) for _ in range(2)]


def _bits(mask):
    """One bit for each value of a 1-D truth tensor, 32 to an int32, the first in the lowest bit."""
    n = mask.numel()
    pad = torch.zeros((n + 31) // 32 * 32, dtype=torch.int64, device=mask.device)
    pad[:n] = mask.long()
    return (pad.view(-1, 32) << torch.arange(32, device=mask.device)).sum(1).to(torch.int32)


def _unbits(bits, n):
    return ((bits[:, None] >> torch.arange(32, device=bits.device)) & 1).flatten()[:n] != 0


def _int(x):
    return torch.as_tensor(x).to(device="cuda", dtype=torch.int32).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "route":
        # a bias of the size that balancing gives: a few hundredths, on scores of (0, 1)
        c.update(logits=(1.5 * _randn(g, c["tokens"], c["experts"])).to(DTYPES[c["x"]]),
                 bias_t=0.05 * _randn(g, c["experts"]) if c["bias"] else None)
    elif c["op"] == "verify":
        n, d, v = c["seqs"], c["drafts"], c["vocab"]
        target = 2.5 * _randn(g, n, d + 1, v)
        # one token of a row stands out, as trained models have it: between a quarter and nine tenths of the whole
        liked = torch.randint(0, v, (n, d + 1, 1), generator=g, device="cuda")
        target.scatter_(2, liked, math.log(v) + 2.0 + 3.5 * _rand(g, n, d + 1, 1))
        near = target[:, :d] + 0.9 * _randn(g, n, d, v)          # a draft model that is right most of the time
        noise = -torch.log(-torch.log(_rand(g, n, d, v).clamp_(1e-20, 1 - 6e-8)))
        tokens = (near + noise if c["draft"] else near).argmax(dim=2) if d else torch.zeros(n, 0, device="cuda")
        if c["temp"] == "mixed":                                 # every fourth request is greedy, the others between 0.6 and 1.2
            temp = 0.6 + 0.6 * _rand(g, n)
            temp[::4] = 0.0
            if d:
                tokens[::4] = near[::4].argmax(dim=2)
        else:
            temp = None
        count = torch.full((n,), d, device="cuda")
        count[3::5] = d // 2                                     # shorter drafts among them
        if c["form"] == "probs":
            target, near = torch.softmax(target, dim=2), torch.softmax(near, dim=2)
        dt = DTYPES[c["x"]]
        c.update(target=target.to(dt).view(n * (d + 1), v), draft_t=near.to(dt).reshape(n * d, v) if c["draft"] else None,
                 tokens=_int(tokens), count=_int(count), u=_rand(g, n, d + 1), temp_t=temp)
    elif c["op"] == "copy":
        k_src, v_src = _pools(g, c, c["pages"], c["layout"])
        k_dst, v_dst = _pools(g, c, c["n"] + 7)
        src = torch.randperm(c["pages"], generator=g, device="cuda")[: c["n"]]
        dst = torch.randperm(c["n"] + 7, generator=g, device="cuda")[: c["n"]]
        c.update(k_src=k_src, v_src=v_src, k_dst=k_dst, v_dst=v_dst, src=_int(src), dst=_int(dst))
    elif c["op"] == "compact":
        k_src, v_src = _pools(g, c, c["pages"])
        k_dst, v_dst = _pools(g, c, c["to_pages"])
        shared = min(c["shared"], c["used"] // 2)
        each = (c["used"] - shared) // c["seqs"]
        cols = shared + each + 3
        perm = torch.randperm(c["pages"], generator=g, device="cuda")
        table = torch.full((c["seqs"], cols), -1, device="cuda")
        table[:, :shared] = perm[:shared]
        table[:, shared: shared + each] = perm[shared: shared + each * c["seqs"]].view(c["seqs"], each)
        ref = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
        ref[perm[: shared]] = c["seqs"]
        ref[perm[shared: c["used"]]] = 1                         # (the last few belong to no row: held elsewhere)
        lens = (shared + each) * c["page"] - torch.arange(c["seqs"], device="cuda") % c["page"]
        c.update(k_src=k_src, v_src=v_src, k_dst=k_dst, v_dst=v_dst, ref=ref, free=_bits(ref == 0), table=_int(table), lens=_int(lens),
                 ref_dst=torch.zeros(c["to_pages"], dtype=torch.int32, device="cuda"),
                 free_dst=_bits(torch.ones(c["to_pages"], dtype=torch.bool, device="cuda")),
                 table_dst=torch.full((c["seqs"], cols), -1, dtype=torch.int32, device="cuda"))
    else:
        _prepare_steps(c, g)
    return c


def _prepare_steps(c, g):
    """The tables before a pass, and the lengths that its two calls of resize set: `down`, then `up`.  A pass ends with the
    lengths it began with, so that every pass has the same work."""
    n, page = c["seqs"], c["page"]
    base = torch.tensor(_lens(c), device="cuda")
    if c["kind"] != "beams":
        base = base[torch.randperm(n, generator=g, device="cuda")]
    if c["kind"] == "drafts":
        up = base + 1 + c["drafts"]
        down = base + 1 + (_rand(g, n) * (c["drafts"] + 1)).long()
    elif c["kind"] == "turnover":
        gone = torch.rand(n, generator=g, device="cuda").argsort() < n // 2
        up, down = base, torch.where(gone, 0, base)
    else:
        group = torch.rand(n // 4, 4, generator=g, device="cuda").argsort(1) + 4 * torch.arange(n // 4, device="cuda")[:, None]
        base = base.view(-1, 4)[:, :1].expand(-1, 4).reshape(n).contiguous()     # beams of one request are equally long
        up, down = base + 1, base.clone()
        down[group[:, 2:].flatten()] = 0
        c.update(src=_int(group[:, :2].flatten()), dst=_int(group[:, 2:].flatten()))
    cols = (int(up.max()) + page - 1) // page + 2
    have = (up + page - 1) // page
    held = torch.arange(cols, device="cuda") < have[:, None]
    own_page = held.clone()
    if c["kind"] == "beams":                                     # whole pages of the common past stand in all four rows
        past = torch.arange(cols, device="cuda") < (base // page)[:, None]
        first = torch.arange(n, device="cuda") % 4 == 0
        own_page &= ~(past & ~first[:, None])
    count = int(own_page.sum())
    c["pages"] = pages = int(count * 1.2) + 2 * n
    table = torch.full((n, cols), -1, device="cuda")
    table[own_page] = torch.randperm(pages, generator=g, device="cuda")[:count]
    if c["kind"] == "beams":
        from_first = table.view(-1, 4, cols)[:, :1].expand(-1, 4, cols).reshape(n, cols)
        table = torch.where(past, from_first, table)
    ref = torch.zeros(pages, dtype=torch.int32, device="cuda")
    ref.index_add_(0, table[held], torch.ones(int(held.sum()), dtype=torch.int32, device="cuda"))
    k, v = _pools(g, c, pages)
    c.update(k_cache=k, v_cache=v, table=_int(table), lens=_int(up), down=_int(down), up=_int(up), ref=ref, free=_bits(ref == 0))


# ------------------------------------------------------------------------- the plain forms

def _choose(x, n):
    """Places of the n largest of a row in order, the lower place first where they are equal."""
    return torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :n]


def _plain_route(c):
    x, t, e = c["logits"].double(), c["tokens"], c["experts"]
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        s = torch.exp(x - x.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    b = s + c["bias_t"].double() if c["bias"] else s
    if c["groups"] > 1:
        size = e // c["groups"]
        group = torch.sort(b.view(t, c["groups"], size), dim=2, descending=True).values[..., : c["top"]].sum(dim=2)
        open_ = torch.zeros(t, c["groups"], dtype=torch.bool, device="cuda").scatter_(1, _choose(group, c["groups_used"]), True)
        b = torch.where(open_.repeat_interleave(size, dim=1), b, float("-inf"))
    ids = _choose(b, c["used"])
    w = s.gather(1, ids)
    if c["normalise"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"ids": ids.int(), "weights": (w * 2.5).float()}


def _plain_verify(c):
    n, d, v = c["seqs"], c["drafts"], c["vocab"]
    p = c["target"].double().view(n, d + 1, v)
    q = c["draft_t"].double().view(n, d, v) if c["draft"] else None
    greedy = torch.zeros(n, dtype=torch.bool, device="cuda")
    if c["form"] == "logits":
        if c["temp_t"] is not None:
            greedy = c["temp_t"] == 0
            t = torch.where(greedy, 1.0, c["temp_t"].double())[:, None, None]
            best = torch.where(p == p.amax(dim=2, keepdim=True), torch.arange(v, device="cuda"), v).amin(dim=2)
            p, q = p / t, q / t if c["draft"] else None
        p = torch.exp(p - p.amax(dim=2, keepdim=True))
        p = p / p.sum(dim=2, keepdim=True)
        if c["draft"]:
            q = torch.exp(q - q.amax(dim=2, keepdim=True))
            q = q / q.sum(dim=2, keepdim=True)
    tok, u, count = c["tokens"].long(), c["u"].double(), c["count"].long()
    at = tok[:, :, None]
    qt = q.gather(2, at)[:, :, 0] if c["draft"] else torch.ones(n, d, dtype=torch.float64, device="cuda")
    yes = u[:, :d] * qt < p[:, :d].gather(2, at)[:, :, 0]
    if c["temp_t"] is not None:
        yes = torch.where(greedy[:, None], tok == best[:, :d], yes)
    yes &= torch.arange(d, device="cuda") < count[:, None]
    took = yes.long().cumprod(dim=1).sum(dim=1)
    row = p[torch.arange(n, device="cuda"), took]
    if d:
        j = took.clamp(max=d - 1)
        if c["draft"]:
            less = q[torch.arange(n, device="cuda"), j]
        else:
            less = torch.zeros(n, v, dtype=torch.float64, device="cuda").scatter_(1, tok.gather(1, j[:, None]), 1.0)
        row = torch.where((took < count)[:, None], (row - less).clamp(min=0), row)
    run_sum = row.cumsum(dim=1)
    last = torch.where(row > 0, torch.arange(v, device="cuda"), 0).amax(dim=1)
    follows = torch.minimum((run_sum <= u[:, d:] * run_sum[:, -1:]).sum(dim=1), last)
    if c["temp_t"] is not None:
        follows = torch.where(greedy, best.gather(1, took[:, None])[:, 0], follows)
    place = torch.arange(d + 1, device="cuda")
    out = torch.cat([tok, follows[:, None]], dim=1)
    out = torch.where(place < took[:, None], out, torch.where(place == took[:, None], follows[:, None], -1))
    return {"tokens": out.int(), "accepted": took.int()}


def _plain_copy(c):
    src, dst = c["src"].long(), c["dst"].long()
    c["k_dst"][dst] = c["k_src"][src]
    c["v_dst"][dst] = c["v_src"][src]
    return {"k": c["k_dst"], "v": c["v_dst"]}


def _plain_compact(c):
    used = ~_unbits(c["free"], c["pages"])
    new = used.long().cumsum(0) - 1
    src = used.nonzero()[:, 0]
    m = src.numel()
    c["k_dst"][:m], c["v_dst"][:m] = c["k_src"][src], c["v_src"][src]
    c["ref_dst"].zero_()
    c["ref_dst"][:m] = c["ref"][src]
    c["free_dst"].copy_(_bits(torch.arange(c["to_pages"], device="cuda") >= m))
    cols = torch.arange(c["table"].shape[1], device="cuda")
    held = cols * c["page"] < c["lens"][:, None]
    c["table_dst"].copy_(torch.where(held, new[c["table"].long().clamp(min=0)], -1))
    return {"k": c["k_dst"], "v": c["v_dst"], "ref": c["ref_dst"], "free": c["free_dst"], "table": c["table_dst"],
            "n_used": used.sum(dtype=torch.int32).view(1)}


def _plain_resize(c, new_lens):
    n, page, pages = c["seqs"], c["page"], c["pages"]
    table, ref, lens, new = c["table"], c["ref"], c["lens"].long(), new_lens.long()
    cols = torch.arange(table.shape[1], device="cuda")
    have, want = (lens + page - 1) // page, (new + page - 1) // page
    # the pages that shrinking sequences leave
    gone = (cols >= want[:, None]) & (cols < have[:, None])
    left = table[gone].long()
    ref.index_add_(0, left, torch.full_like(left, -1, dtype=torch.int32))
    free = _unbits(c["free"], pages)
    free[left] = ref[left] == 0
    table[gone] = -1
    # a sequence that grows inside a page that others hold gets a copy; where all holders do, the first keeps the page
    seq = torch.arange(n, device="cuda")
    tail = table[seq, (have - 1).clamp(min=0)].long().clamp(min=0)
    copies = (new > lens) & (lens % page != 0) & (ref[tail] > 1)
    holders = torch.zeros(pages, dtype=torch.int64, device="cuda").index_add_(0, tail, copies.long())
    first = torch.full((pages,), n, device="cuda").scatter_reduce_(0, tail, torch.where(copies, seq, n), "amin")
    stays = copies & (holders[tail] == ref[tail]) & (first[tail] == seq)
    copies &= ~stays
    need = (want - have).clamp(min=0) + copies.long()
    end = need.cumsum(0)
    missing = (end[-1] - free.sum()).clamp(min=0)
    grown = (new > lens) & (missing == 0)
    copies &= missing == 0
    # free pages are taken in the order of their numbers
    order = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    order.scatter_(0, torch.where(free, free.long().cumsum(0) - 1, pages), torch.arange(pages, device="cuda"))
    fresh = grown[:, None] & (cols >= have[:, None]) & (cols < want[:, None])
    place = (end - need + copies)[:, None] + cols - have[:, None]
    table[fresh] = order[place[fresh]].int()
    at = copies.nonzero()[:, 0]
    mine = order[(end - need)[at]]
    old, rows = tail[at], lens[at] % page
    some = (torch.arange(page, device="cuda") < rows[:, None])[:, None, :, None]
    for pool in (c["k_cache"], c["v_cache"]):
        pool[mine] = torch.where(some, pool[old], pool[mine])
    table[at, have[at] - 1] = mine.int()
    ref.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    taken = torch.cat([table[fresh].long(), mine])
    ref[taken] = 1
    free[taken] = False
    c["lens"].copy_(torch.where((new < lens) | grown, new, lens))
    c["free"].copy_(_bits(free))
    return missing.int().view(1)


def _plain_fork(c):
    n, page, pairs = c["seqs"], c["page"], c["src"].numel()
    table, lens, src, dst = c["table"], c["lens"], c["src"].long(), c["dst"].long()
    cols = torch.arange(table.shape[1], device="cuda")
    length = lens[src]
    fits = (src != dst) & (lens[dst] == 0)
    pair = torch.arange(pairs, device="cuda")
    first = torch.full((n,), pairs, device="cuda").scatter_reduce_(0, dst, torch.where(fits, pair, pairs), "amin")
    fits &= first[dst] == pair
    shared = fits[:, None] & (cols * page < length[:, None])
    rows = table[src]
    table[dst[:, None].expand_as(rows)[shared], cols.expand_as(rows)[shared]] = rows[shared]
    pages = rows[shared].long()
    c["ref"].index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    lens.scatter_add_(0, dst, torch.where(fits, length, 0))


def _state_of_steps(c, *missing):
    return {"k": c["k_cache"], "v": c["v_cache"], "table": c["table"], "lens": c["lens"], "ref": c["ref"], "free": c["free"],
            "missing": list(missing)}


def _plain_steps(c):
    a = _plain_resize(c, c["down"])
    if c["kind"] == "beams":
        _plain_fork(c)
    return _state_of_steps(c, a, _plain_resize(c, c["up"]))


# ------------------------------------------------------------------------------ one pass

def run(state):
    c = state
    if not own:
        return {"route": _plain_route, "verify": _plain_verify, "copy": _plain_copy, "compact": _plain_compact,
                "steps": _plain_steps}[c["op"]](c)
    from ternary_bit_quantized_amd import q2_0 as B
    if c["op"] == "route":
        score = B.Q2_0_SCORE_SIGMOID if c["score"] == "sigmoid" else B.Q2_0_SCORE_SOFTMAX
        ids, weights = B.q2_0_moe_route_groups(c["logits"], c["used"], score, bias=c["bias_t"], n_group=c["groups"],
                                               n_group_used=c["groups_used"], group_top=c["top"], normalise=c["normalise"], scale=2.5)
        return {"ids": ids, "weights": weights}
    if c["op"] == "verify":
        form = B.Q2_0_DRAFT_PROBS if c["form"] == "probs" else B.Q2_0_DRAFT_LOGITS
        tokens, accepted = B.q2_0_draft_verify(c["target"], c["draft_t"], c["tokens"], c["count"], c["u"], form=form,
                                               temperature=c["temp_t"])
        return {"tokens": tokens, "accepted": accepted}
    if c["op"] == "copy":
        B.q2_0_kv_copy(c["k_dst"], c["v_dst"], c["k_src"], c["v_src"], c["src"], c["dst"])
        return {"k": c["k_dst"], "v": c["v_dst"]}
    if c["op"] == "compact":
        n_used = B.q2_0_kv_compact(c["k_dst"], c["v_dst"], c["ref_dst"], c["free_dst"], c["table_dst"], c["k_src"], c["v_src"],
                                   c["ref"], c["free"], c["table"], c["lens"])
        return {"k": c["k_dst"], "v": c["v_dst"], "ref": c["ref_dst"], "free": c["free_dst"], "table": c["table_dst"], "n_used": n_used}
    a = B.q2_0_kv_resize(c["k_cache"], c["v_cache"], c["ref"], c["free"], c["table"], c["lens"], c["down"])
    if c["kind"] == "beams":
        B.q2_0_kv_fork(c["ref"], c["table"], c["page"], c["lens"], c["src"], c["dst"])
    b = B.q2_0_kv_resize(c["k_cache"], c["v_cache"], c["ref"], c["free"], c["table"], c["lens"], c["up"])
    return _state_of_steps(c, a, b)


# ------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    c = prepare(case, seed)
    return {"route": _exact_route, "verify": _exact_verify, "copy": _exact_copy, "compact": _exact_compact,
            "steps": _exact_steps}[c["op"]](c)


def _exact_route(c):
    x = c["logits"].double()
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1)
    b = s if c["bias_t"] is None else s + c["bias_t"].double()[None]
    size = c["experts"] // c["groups"]
    parts = b.split(size, dim=1)
    value = torch.stack([part.topk(min(c["top"], size), dim=1).values.sum(dim=1) for part in parts], dim=1)
    rank = torch.argsort(torch.argsort(-value, dim=1, stable=True), dim=1)
    b = torch.cat([torch.where(rank[:, g: g + 1] < c["groups_used"], part, -float("inf")) for g, part in enumerate(parts)], dim=1)
    ids = torch.argsort(-b, dim=1, stable=True)[:, : c["used"]]
    w = torch.gather(s, 1, ids)
    return {"ids": ids.int(), "weights": 2.5 * w / (w.sum(dim=1, keepdim=True) if c["normalise"] else 1.0)}


def _exact_verify(c):
    n, d, v = c["seqs"], c["drafts"], c["vocab"]
    tokens, count, u = c["tokens"].tolist(), c["count"].tolist(), c["u"].double().tolist()
    temp = [1.0] * n if c["temp_t"] is None else c["temp_t"].double().tolist()

    def probabilities(row, t):
        row = row.double()
        if c["form"] == "probs":
            return row
        if t == 0:
            best = int((row == row.max()).nonzero()[0])
            return torch.zeros_like(row).index_fill_(0, torch.tensor([best], device=row.device), 1.0)
        return torch.softmax(row / t, dim=0)

    out = torch.full((n, d + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(n, dtype=torch.int32)
    for s in range(n):
        for j in range(count[s] + 1):
            p = probabilities(c["target"][s * (d + 1) + j], temp[s])
            if j < count[s]:
                t = tokens[s][j]
                if c["draft"]:
                    q = probabilities(c["draft_t"][s * d + j], temp[s])
                else:
                    q = torch.zeros_like(p)
                    q[t] = 1.0
                if temp[s] == 0:
                    took, left = bool(p[t] > 0), p
                else:
                    took, left = u[s][j] * float(q[t]) < float(p[t]), torch.relu(p - q)
                if took:
                    out[s, j] = t
                    continue
                p = left
            sums = torch.cumsum(p, dim=0)
            at = int(torch.searchsorted(sums, sums[-1:] * u[s][d], right=True))
            out[s, j] = min(at, int(p.nonzero()[-1]))
            accepted[s] = j
            break
    return {"tokens": out, "accepted": accepted}


def _exact_copy(c):
    k, v = c["k_dst"].double(), c["v_dst"].double()
    for a, b in zip(c["src"].tolist(), c["dst"].tolist()):
        k[b], v[b] = c["k_src"][a].double(), c["v_src"][a].double()
    return {"k": k, "v": v}


def _set_of(bits, n):
    words = [w & 0xFFFFFFFF for w in bits.tolist()]
    return {i for i in range(n) if words[i // 32] >> (i % 32) & 1}


def _words_of(pages, n):
    words = [0] * ((n + 31) // 32)
    for i in pages:
        words[i // 32] |= 1 << (i % 32)
    return torch.tensor([w - (1 << 32) if w >> 31 else w for w in words], dtype=torch.int32)


def _exact_compact(c):
    free = _set_of(c["free"], c["pages"])
    k, v, ref = c["k_dst"].double(), c["v_dst"].double(), [0] * c["to_pages"]
    count, number = c["ref"].tolist(), {}
    for page in range(c["pages"]):
        if page not in free:
            at = number[page] = len(number)
            k[at], v[at], ref[at] = c["k_src"][page].double(), c["v_src"][page].double(), count[page]
    table = [[number[p] if i * c["page"] < length else -1 for i, p in enumerate(row)]
             for row, length in zip(c["table"].tolist(), c["lens"].tolist())]
    return {"k": k, "v": v, "ref": torch.tensor(ref, dtype=torch.int32), "table": torch.tensor(table, dtype=torch.int32),
            "free": _words_of(range(len(number), c["to_pages"]), c["to_pages"]), "n_used": torch.tensor([len(number)], dtype=torch.int32)}


def _exact_steps(c):
    page, n = c["page"], c["seqs"]
    table, lens, ref = c["table"].tolist(), c["lens"].tolist(), c["ref"].tolist()
    free = _set_of(c["free"], c["pages"])
    pools = [c["k_cache"].double(), c["v_cache"].double()]

    def resize(new):
        for s in range(n):
            for i in range(-(-new[s] // page), -(-lens[s] // page)):
                p, table[s][i] = table[s][i], -1
                ref[p] -= 1
                if ref[p] == 0:
                    free.add(p)
            lens[s] = min(lens[s], new[s])
        holds = {}
        for s in range(n):
            if new[s] > lens[s] and lens[s] % page:
                holds.setdefault(table[s][lens[s] // page], []).append(s)
        copied = {s for p, who in holds.items() if ref[p] > 1 for s in (who[1:] if len(who) == ref[p] else who)}
        need = sum(-(-new[s] // page) - -(-lens[s] // page) + (s in copied) for s in range(n) if new[s] > lens[s])
        missing = max(0, need - len(free))
        heap = iter(sorted(free))
        for s in range(n):
            if missing or new[s] <= lens[s]:
                continue
            if s in copied:
                i, mine = lens[s] // page, next(heap)
                old, table[s][i] = table[s][i], mine
                for pool in pools:
                    pool[mine, :, : lens[s] % page] = pool[old, :, : lens[s] % page]
                ref[old] -= 1
                ref[mine] = 1
                free.remove(mine)
            for i in range(-(-lens[s] // page), -(-new[s] // page)):
                table[s][i] = next(heap)
                ref[table[s][i]] = 1
                free.remove(table[s][i])
            lens[s] = new[s]
        return torch.tensor([missing], dtype=torch.int32)

    a = resize(c["down"].tolist())
    if c["kind"] == "beams":
        for s, t in zip(c["src"].tolist(), c["dst"].tolist()):
            for i in range(-(-lens[s] // page)):
                table[t][i] = table[s][i]
                ref[table[s][i]] += 1
            lens[t] = lens[s]
    b = resize(c["up"].tolist())
    return {"k": pools[0], "v": pools[1], "table": torch.tensor(table, dtype=torch.int32), "lens": torch.tensor(lens, dtype=torch.int32),
            "ref": torch.tensor(ref, dtype=torch.int32), "free": _words_of(free, c["pages"]), "missing": [a, b]}
