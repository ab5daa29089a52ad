"""The decoder-layer operators around the Q2_0 products, as cases to time and compare.

Four operators of one decode (or prompt) step over Q2_0 weights:

  append   position rotation of q and k, and the store of k and v into a paged cache
  attn     attention of a batch of sequences over that cache, with a prefix they share
  route    expert choice: the n_used largest of a token's router logits, and their weights
  moe      a whole expert layer for a few tokens: gate, up, SiLU, down and the weighted sum

`run` computes an operator in plain 32-bit torch operations, or (own = True) through the
package's entry points; `exact` computes it in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one sequence goes into the cache: 4096-wide q, 1024-wide k and v, heads of 128
        dict(name="append_decode_1", op="append", tokens=1, seqs=1, n_q=32, n_kv=8, dim=128, rot=128, style="half",
             x="f32", cache="bf16", page=16, start=777),
        # a prompt batch of ragged length, four sequences of a serving step at once
        dict(name="append_prompt_4099", op="append", tokens=4099, seqs=4, n_q=32, n_kv=8, dim=128, rot=128, style="half",
             x="f32", cache="bf16", page=64, start=0),
        # a single sequence's decode step early in a chat: latency counts
        dict(name="attn_one_777", op="attn", seqs=1, n_qt=1, prefix=0, own_lo=777, own_hi=777, n_q=32, n_kv=8, dim=128,
             cache="bf16", page=16),
        # an ordinary serving batch under one system prompt, ragged own parts
        dict(name="attn_batch_16", op="attn", seqs=16, n_qt=1, prefix=4096, own_lo=65, own_hi=513, n_q=32, n_kv=8, dim=128,
             cache="bf16", page=16),
        # four draft tokens per sequence to verify, 64-wide heads, seven query heads to a key head, a
        # prefix that ends inside a page
        dict(name="attn_draft_8x4", op="attn", seqs=8, n_qt=4, prefix=1001, own_lo=5, own_hi=301, n_q=14, n_kv=2, dim=64,
             cache="f16", page=24),
        # a large batch over one long document
        dict(name="attn_doc_64", op="attn", seqs=64, n_qt=1, prefix=32768, own_lo=1, own_hi=1025, n_q=32, n_kv=8, dim=128,
             cache="bf16", page=64),
        # the router of one token, and of a prompt batch (128 experts, 8 used)
        dict(name="route_1", op="route", tokens=1, experts=128, used=8, x="f32", normalise=True),
        dict(name="route_4096", op="route", tokens=4096, experts=128, used=8, x="f32", normalise=True),
        # the benchmark's expert layer (128 experts of 768 x 2048, 8 per token) for one token
        dict(name="moe_1", op="moe", tokens=1, experts=128, used=8, ff=768, hidden=2048, x="f32"),
        # fewer, other experts with rows of an odd number of blocks, 16-bit activations
        dict(name="moe_5_odd", op="moe", tokens=5, experts=60, used=4, ff=704, hidden=1600, x="bf16"),
        # a small and the largest serving batch through the benchmark's expert layer
        dict(name="moe_16", op="moe", tokens=16, experts=128, used=8, ff=768, hidden=2048, x="f32"),
        dict(name="moe_64", op="moe", tokens=64, experts=128, used=8, ff=768, hidden=2048, x="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "route", "moe", "moe"])
    if op == "append":
        dim = rng.choice([64, 128, 256])
        n_kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 4, 7, 8]) if dim < 256 else rng.choice([1, 2])
        seqs = _log(rng, 1, 32)
        return dict(op=op, tokens=max(seqs, _log(rng, 1, 2000)) | 1, seqs=seqs, n_q=n_kv * min(group, 32 // n_kv), n_kv=n_kv,
                    dim=dim, rot=rng.choice([dim, dim // 2]), style=rng.choice(["half", "pairs"]),
                    x=rng.choice(["f32", "bf16", "f16"]), cache=rng.choice(["bf16", "f16"]), page=rng.choice([16, 20, 64]),
                    start=_log(rng, 1, 8000))
    if op == "attn":
        dim = rng.choice([64, 128, 128, 256])
        n_kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 8])
        seqs = _log(rng, 1, 64)
        own_lo = _log(rng, 1, 100)
        longest = min(16000, 32768 * 64 * 128 // (4 * seqs * dim))          # within the largest listed case
        return dict(op=op, seqs=seqs, n_qt=rng.choice([1, 1, 1, 2, 3]), prefix=rng.choice([0, _log(rng, 33, longest) | 1]),
                    own_lo=own_lo, own_hi=own_lo + 2 * _log(rng, 1, 500), n_q=n_kv * min(group, 32 // n_kv), n_kv=n_kv, dim=dim,
                    cache=rng.choice(["bf16", "f16"]), page=rng.choice([16, 24, 64, 128]))
    if op == "route":
        experts = rng.choice([8, 60, 64, 128, 160, 256, 384])
        return dict(op=op, tokens=_log(rng, 1, 4000) | 1, experts=experts, used=rng.randint(1, 8), x=rng.choice(["f32", "bf16", "f16"]),
                    normalise=rng.choice([True, False]))
    ff, hidden = 64 * rng.randint(4, 24), 64 * rng.randint(8, 32)
    most = min(64, 64 * 768 * 2048 // (ff * hidden))                        # likewise
    return dict(op=op, tokens=_log(rng, 1, most), experts=rng.choice([8, 16, 60, 64, 100, 128]), used=rng.randint(1, 8),
                ff=ff, hidden=hidden, x=rng.choice(["f32", "bf16", "f16"]))


# ----------------------------------------------------------------------- sizes of a case

def _own_lens(c):
    """Own lengths of the sequences, spread evenly over [own_lo, own_hi]."""
    n = c["seqs"]
    return [c["own_lo"] + (c["own_hi"] - c["own_lo"]) * i // max(1, n - 1) for i in range(n)]


def _append_counts(c):
    """Tokens of each sequence in an append call: as even as the count allows, at least one."""
    n, t = c["seqs"], c["tokens"]
    return [t // n + (1 if i < t % n else 0) for i in range(n)]


def _size(name):
    return {"f32": 4, "f16": 2, "bf16": 2}[name]


def work(case):
    c = case
    if c["op"] == "append":
        row_in = (c["n_q"] + 2 * c["n_kv"]) * c["dim"] * _size(c["x"])
        row_out = (c["n_q"] + 2 * c["n_kv"]) * c["dim"] * 2
        # a rotation is two multiply-adds per element of q and k
        return {"bytes": c["tokens"] * (row_in + row_out + c["rot"] * 4 + 12),
                "flops": c["tokens"] * (c["n_q"] + c["n_kv"]) * c["rot"] * 3}
    if c["op"] == "attn":
        lens = _own_lens(c)
        keys = c["prefix"] + sum(lens)                              # each key and value once
        pairs = sum(c["prefix"] + n for n in lens) * c["n_qt"]      # (query token, key)
        io = 2 * c["seqs"] * c["n_qt"] * c["n_q"] * c["dim"] * 2
        return {"bytes": keys * c["n_kv"] * c["dim"] * 2 * 2 + io + 4 * keys // c["page"],
                "flops": 4 * pairs * c["n_q"] * c["dim"]}
    if c["op"] == "route":
        return {"bytes": c["tokens"] * (c["experts"] * _size(c["x"]) + c["used"] * 8), "flops": c["tokens"] * c["experts"] * 4}
    # every expert that is met once (its expected number for independent choices), 18 bytes per 64 weights
    met = c["experts"] * (1 - (1 - min(1, c["used"] / c["experts"])) ** c["tokens"])
    per = 3 * c["ff"] * c["hidden"]
    return {"bytes": met * per * 18 / 64 + c["tokens"] * (c["hidden"] * (_size(c["x"]) + 4) + c["used"] * 8),
            "flops": 2 * c["tokens"] * c["used"] * per}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _q2_0(g, experts, rows, k):
    """Seeded ternary Q2_0 matrices, one after the other: (experts, rows, k/64*18) bytes."""
    blocks = experts * rows * (k // 64)
    t = torch.randint(0, 81, (blocks, 16), generator=g, device="cuda", dtype=torch.uint8)
    lut = torch.tensor([(v % 3) | (v // 3 % 3) << 2 | (v // 9 % 3) << 4 | (v // 27) << 6 for v in range(81)],
                       dtype=torch.uint8, device="cuda")
    d = torch.empty(blocks, 1, device="cuda").uniform_(0.005, 0.05, generator=g).to(torch.float16)
    out = torch.empty(blocks, 18, dtype=torch.uint8, device="cuda")
    out[:, :2] = d.view(torch.uint8)
    out[:, 2:] = lut[t.int()]
    return out.view(experts, rows, (k // 64) * 18)


def _rope_table(n_pos, rot):
    """cos and sin of position times the usual geometric frequencies, (n_pos, rot) f32."""
    f = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _choose(logits, used):
    """The `used` largest logits of a row in order, the lower index first where they are equal."""
    return torch.sort(logits, dim=-1, descending=True, stable=True).indices[..., :used]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "append":
        t, counts, page = c["tokens"], _append_counts(c), c["page"]
        seq = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(counts)).int().cuda()
        pos = torch.cat([c["start"] + torch.arange(n) for n in counts]).int().cuda()
        cols = (c["start"] + max(counts) + page - 1) // page
        first = c["start"] // page
        held = cols - first                        # pages of a sequence that the call can write
        n_pages = c["seqs"] * held
        perm = torch.randperm(n_pages, generator=g, device="cuda").int().view(c["seqs"], held)
        table = torch.zeros(c["seqs"], cols, dtype=torch.int32, device="cuda")
        table[:, first:] = perm
        shape = (n_pages, c["n_kv"], page, c["dim"])
        c.update(seq=seq, pos=pos, table=table,
                 k_cache=_randn(g, *shape).to(DTYPES[c["cache"]]), v_cache=_randn(g, *shape).to(DTYPES[c["cache"]]),
                 q=_randn(g, t, c["n_q"] * c["dim"]).to(DTYPES[c["x"]]),
                 k=_randn(g, t, c["n_kv"] * c["dim"]).to(DTYPES[c["x"]]),
                 v=_randn(g, t, c["n_kv"] * c["dim"]).to(DTYPES[c["x"]]),
                 rope=_rope_table(c["start"] + max(counts), c["rot"]))
    elif c["op"] == "attn":
        page, n, pre = c["page"], c["seqs"], c["prefix"]
        order = torch.randperm(n, generator=g, device="cuda")
        lens = (pre + torch.tensor(_own_lens(c), device="cuda")[order]).int()
        max_len = pre + c["own_hi"]
        cols, shared = (max_len + page - 1) // page, pre // page
        n_pages = shared + n * (cols - shared)
        perm = torch.randperm(n_pages, generator=g, device="cuda").int()
        table = torch.empty(n, cols, dtype=torch.int32, device="cuda")
        table[:, :shared] = perm[:shared]
        table[:, shared:] = perm[shared:].view(n, cols - shared)
        dt = DTYPES[c["cache"]]
        shape = (n_pages, c["n_kv"], page, c["dim"])
        k, v = _randn(g, *shape).to(dt), _randn(g, *shape).to(dt)
        if pre % page:                             # the prefix ends inside a page: every sequence has its copy
            edge = table[:, shared].long()
            for t in (k, v):
                t[edge, :, : pre % page] = t[edge[0], :, : pre % page].clone()
        # queries with the spread that gives scores of a few units, as trained heads have
        q = (1.5 * _randn(g, n * c["n_qt"], c["n_q"] * c["dim"])).to(dt)
        c.update(table=table, lens=lens, max_len=max_len, k_cache=k, v_cache=v, q=q, scale=1.0 / math.sqrt(c["dim"]))
    elif c["op"] == "route":
        c.update(logits=(2.0 * _randn(g, c["tokens"], c["experts"])).to(DTYPES[c["x"]]))
    else:
        e, f, h = c["experts"], c["ff"], c["hidden"]
        logits = 2.0 * _randn(g, c["tokens"], e)
        ids = _choose(logits, c["used"])
        c.update(w_gate=_q2_0(g, e, f, h), w_up=_q2_0(g, e, f, h), w_down=_q2_0(g, e, h, f),
                 ids=ids.int().contiguous(), weights=torch.softmax(logits.gather(1, ids), dim=1).contiguous(),
                 act=_randn(g, c["tokens"], h).to(DTYPES[c["x"]]))
    return c


# ------------------------------------------------------------- the plain forms, in 32 bits

def _rotate(x, cos, sin, rot, style):
    """x (tokens, heads, dim): its first rot elements turned by the table's angles."""
    r, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if style == "half":
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([r, rest], dim=-1)


def _plain_append(c):
    t, d, rot, page = c["tokens"], c["dim"], c["rot"], c["page"]
    pos, seq = c["pos"].long(), c["seq"].long()
    turn = c["rope"][pos]
    cos, sin = turn[:, : rot // 2], turn[:, rot // 2:]
    q = _rotate(c["q"].float().view(t, -1, d), cos, sin, rot, c["style"])
    k = _rotate(c["k"].float().view(t, -1, d), cos, sin, rot, c["style"])
    where, off = c["table"][seq, pos // page].long(), pos % page
    c["k_cache"][where, :, off] = k.to(c["k_cache"].dtype)
    c["v_cache"][where, :, off] = c["v"].float().view(t, -1, d).to(c["v_cache"].dtype)
    return {"q": q.to(c["k_cache"].dtype).view(t, -1), "k_cache": c["k_cache"], "v_cache": c["v_cache"]}


def _gather(cache, table, at, page):
    """Keys or values `at` (positions) of each row of `table`: (rows, kv heads, positions, dim) f32."""
    return cache[table[:, at // page].long(), :, at % page].float().permute(0, 2, 1, 3).contiguous()


def _plain_attn(c):
    n, nt, kv, d, page, pre = c["seqs"], c["n_qt"], c["n_kv"], c["dim"], c["page"], c["prefix"]
    grp = c["n_q"] // kv
    q = c["q"].float().view(n, nt, kv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, kv, nt * grp, d) * c["scale"]
    at = torch.arange(pre, c["max_len"], device="cuda")
    k, v = _gather(c["k_cache"], c["table"], at, page), _gather(c["v_cache"], c["table"], at, page)
    s = q @ k.transpose(2, 3).contiguous()                                  # (n, kv, rows, own)
    last = c["lens"].long()[:, None] - nt + 1 + torch.arange(nt, device="cuda")   # keys a query may see
    seen = at < last.repeat_interleave(grp, dim=1)[:, None, :, None]
    s = torch.where(seen, s, float("-inf"))
    top = s.amax(dim=3, keepdim=True)
    if pre:                                                                 # the shared keys once for all rows
        p_at = torch.arange(pre, device="cuda")
        pk = _gather(c["k_cache"], c["table"][:1], p_at, page)[0]
        pv = _gather(c["v_cache"], c["table"][:1], p_at, page)[0]
        rows = q.transpose(0, 1).reshape(kv, n * nt * grp, d)
        ps = (rows @ pk.transpose(1, 2).contiguous()).view(kv, n, nt * grp, pre).transpose(0, 1)
        ps = torch.where(p_at < last.repeat_interleave(grp, dim=1)[:, None, :, None], ps, float("-inf"))
        top = torch.maximum(top, ps.amax(dim=3, keepdim=True))
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total, o = p.sum(dim=3, keepdim=True), p @ v
    if pre:
        pp = torch.exp(ps - top)
        total = total + pp.sum(dim=3, keepdim=True)
        o = o + (pp.transpose(0, 1).reshape(kv, -1, pre) @ pv).view(kv, n, nt * grp, d).transpose(0, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.view(n, kv, nt, grp, d).permute(0, 2, 1, 3, 4).reshape(n * nt, -1).to(c["q"].dtype)


def _plain_route(c):
    x = c["logits"].float()
    ids = _choose(x, c["used"])
    p = torch.exp(x - x.amax(dim=1, keepdim=True))
    w = p.gather(1, ids)
    return {"ids": ids.int(), "weights": w / (w if c["normalise"] else p).sum(dim=1, keepdim=True)}


def _decode(w):
    """f32 values of Q2_0 rows: (..., blocks*18) bytes -> (..., blocks*64)."""
    b = w.view(*w.shape[:-1], -1, 18)
    d = b[..., :2].contiguous().view(torch.float16).float()
    shift = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=w.device)
    q = ((b[..., 2:, None] >> shift) & 3).flatten(-2)
    return ((q.float() - 1.0) * d).flatten(-2)


def _plain_moe(c):
    ids = c["ids"].long().flatten()
    x = c["act"].float().repeat_interleave(c["used"], dim=0)[:, :, None]
    gate, up = _decode(c["w_gate"][ids]) @ x, _decode(c["w_up"][ids]) @ x
    h = gate * (1.0 / (1.0 + torch.exp(-gate))) * up
    y = (_decode(c["w_down"][ids]) @ h).view(c["tokens"], c["used"], -1)
    return (c["weights"][:, :, None] * y).sum(dim=1)


# ------------------------------------------------------------------------------ one pass

def run(state):
    c = state
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "route": _plain_route, "moe": _plain_moe}[c["op"]](c)
    from ternary_bit_quantized_amd import q2_0 as B
    if c["op"] == "append":
        style = B.Q2_0_ROPE_HALF if c["style"] == "half" else B.Q2_0_ROPE_PAIRS
        q = B.q2_0_kv_append(c["k_cache"], c["v_cache"], c["table"], c["seq"], c["pos"], c["k"], c["v"], rope=c["rope"],
                             style=style, q=c["q"])
        return {"q": q, "k_cache": c["k_cache"], "v_cache": c["v_cache"]}
    if c["op"] == "attn":
        return B.q2_0_attn_shared(c["q"], c["k_cache"], c["v_cache"], c["table"], c["lens"], c["scale"],
                                  prefix_len=c["prefix"], max_len=c["max_len"], n_qt=c["n_qt"])
    if c["op"] == "route":
        ids, weights = B.q2_0_moe_route(c["logits"], c["used"], normalise=c["normalise"])
        return {"ids": ids, "weights": weights}
    return B.q2_0_moe_layer(c["w_gate"], c["w_up"], c["w_down"], c["experts"], c["ff"], c["hidden"], c["act"], c["ids"],
                            c["weights"])


# ------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    c = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "route": _exact_route, "moe": _exact_moe}[c["op"]](c)


def _exact_append(c):
    rot, d = c["rot"], c["dim"]
    half = rot // 2
    e = torch.arange(half, device="cuda")
    i, j = (e, e + half) if c["style"] == "half" else (2 * e, 2 * e + 1)     # the elements of each turned pair
    turn = c["rope"].double()[c["pos"].long()]
    z = torch.complex(turn[:, :half], turn[:, half:])[:, None]

    def turned(x):
        y = x.double().view(c["tokens"], -1, d).clone()
        w = torch.complex(y[..., i], y[..., j]) * z
        y[..., i], y[..., j] = w.real.contiguous(), w.imag.contiguous()
        return y

    kc, vc = c["k_cache"].double(), c["v_cache"].double()
    k, v = turned(c["k"]), c["v"].double().view(c["tokens"], -1, d)
    slot = (c["table"][c["seq"].long(), (c["pos"] // c["page"]).long()] * c["page"] + c["pos"] % c["page"]).long()
    for cache, new in ((kc, k), (vc, v)):
        flat = cache.transpose(1, 2).reshape(-1, c["n_kv"], d).clone()
        flat[slot] = new
        cache.copy_(flat.view(cache.shape[0], c["page"], c["n_kv"], d).transpose(1, 2))
    return {"q": turned(c["q"]).view(c["tokens"], -1), "k_cache": kc, "v_cache": vc}


def _exact_attn(c):
    nt, kv, d, grp = c["n_qt"], c["n_kv"], c["dim"], c["n_q"] // c["n_kv"]
    out = torch.zeros(c["seqs"], nt, kv, grp, d, dtype=torch.float64, device="cuda")
    q = c["q"].double().view(c["seqs"], nt, kv, grp, d)
    for s, length in enumerate(c["lens"].tolist()):
        pages = c["table"][s].long()
        k = c["k_cache"][pages].double().transpose(1, 2).reshape(-1, kv, d)[:length]
        v = c["v_cache"][pages].double().transpose(1, 2).reshape(-1, kv, d)[:length]
        for j in range(nt):
            keys = length - nt + 1 + j
            if keys > 0:
                score = torch.einsum("hgd,lhd->hgl", q[s, j], k[:keys]) * c["scale"]
                out[s, j] = torch.einsum("hgl,lhd->hgd", torch.softmax(score, dim=2), v[:keys])
    return out.view(c["seqs"] * nt, -1)


def _exact_route(c):
    x = c["logits"].double()
    ids = torch.argsort(-x, dim=1, stable=True)[:, : c["used"]]
    chosen = x.gather(1, ids)
    w = torch.softmax(chosen, dim=1) if c["normalise"] else torch.exp(chosen - torch.logsumexp(x, dim=1, keepdim=True))
    return {"ids": ids.int(), "weights": w}


def _exact_moe(c):
    value = torch.tensor([-1.0, 0.0, 1.0, 2.0], dtype=torch.float64, device="cuda")

    def matrix(w):
        b = w.view(w.shape[0], -1, 18)
        d = b[:, :, :2].contiguous().view(torch.float16).double()
        codes = torch.stack([value[(b[:, :, 2:] // 4 ** i % 4).long()] for i in range(4)], dim=-1)
        return (codes.flatten(2) * d).flatten(1)

    y = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
    x, ids = c["act"].double(), c["ids"].tolist()
    for e in sorted({e for row in ids for e in row}):
        gate, up, down = matrix(c["w_gate"][e]), matrix(c["w_up"][e]), matrix(c["w_down"][e])
        for t, row in enumerate(ids):
            for u, met in enumerate(row):
                if met == e:
                    a = gate @ x[t]
                    y[t] += c["weights"][t, u].double() * (down @ (a * torch.sigmoid(a) * (up @ x[t])))
    return y
