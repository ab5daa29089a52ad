"""Verification of drafted tokens against the definition in 64 bits: every output is a whole number and has to be the same."""

import numpy as np
import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

FORM = {"logits": B.Q2_0_DRAFT_LOGITS, "probs": B.Q2_0_DRAFT_PROBS}


def types():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def probabilities(row, form, t):
    if form == "probs":
        return row
    if np.isnan(row).any() or np.isposinf(row).any() or np.isneginf(row).all() or not t >= 0:
        return np.full_like(row, np.nan)
    if t == 0:
        return np.eye(1, len(row), int(row.argmax()))[0]
    with np.errstate(all="ignore"):
        e = np.exp((row - row.max()) / min(max(t, 2.0 ** -100), 2.0 ** 100))     # (the documented ends)
    return e / e.sum()


def drawn(w, u):
    w = np.where(w <= 0, 0, w)
    sums = np.cumsum(w)
    if not (sums[-1] > 0 and np.isfinite(sums[-1])):
        return -1
    over = np.nonzero(sums > max(u, 0.0) * sums[-1])[0]
    return int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])


def reference(target, draft, tokens, n_draft, u, form="logits", temp=None):
    n, most = tokens.shape
    v = target.shape[1]
    out, acc = np.full((n, most + 1), -1, np.int64), np.zeros(n, np.int64)
    for s in range(n):
        nd, t = int(n_draft[s]), 1.0 if temp is None else float(temp[s])
        if not 0 <= nd <= most:
            continue
        greedy = t == 0 and form == "logits"
        for j in range(nd + 1):
            p = probabilities(target[s * (most + 1) + j], form, t)
            if j == nd:
                out[s, j], acc[s] = drawn(p, u[s, most]), j
                break
            tok = int(tokens[s, j])
            known = 0 <= tok < v
            q = np.zeros(v)
            if draft is None:
                q[tok if known else []] = 1.0
            elif not greedy:
                q = probabilities(draft[s * most + j], form, t)
            if known and (p[tok] > 0 if greedy else u[s, j] * q[tok] < p[tok]):
                out[s, j] = tok
                continue
            if greedy:
                left = p
            else:
                left = np.maximum(p - q, 0) if draft is not None else np.where(q > 0, 0, p)
                if left.sum() < 2.0 ** -32:     # next to nothing: rounding alone
                    left = p
            out[s, j], acc[s] = drawn(left, u[s, most]), j
            break
    return out, acc


def check(target, draft, tokens, n_draft, u, form="logits", temp=None, **kw):
    import torch
    out, acc = B.q2_0_draft_verify(target, draft, tokens, n_draft, u, form=FORM[form], temperature=temp, **kw)
    torch.cuda.synchronize()

    def host(t):
        return None if t is None else t.double().cpu().numpy()

    rout, racc = reference(host(target), host(draft), host(tokens), host(n_draft), host(u), form, host(temp))
    assert np.array_equal(acc.cpu().numpy(), racc), (acc.cpu().numpy(), racc)
    assert np.array_equal(out.cpu().numpy(), rout), (out.cpu().numpy(), rout)
    return out, acc


def rows(g, n, v, x, pad=0, off=0, spread=2.5):
    import torch
    buf = (spread * torch.randn(n * (v + pad) + off, generator=g, device="cuda")).to(types()[x])
    return buf[off:].view(n, v + pad)[:, :v]


def case(n, most, v, x="f32", form="logits", has_draft=True, seed=0, pad=0, off=0):
    """Rows in which one token stands out, drafts drawn from the draft's rows (or the target's best tokens)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    target = rows(g, n * (most + 1), v, x, pad, off)
    liked = torch.randint(0, v, (n * (most + 1), 1), generator=g, device="cuda")
    target.scatter_(1, liked, float(np.log(v) + 4.0))
    near = (target.float().reshape(n, most + 1, v)[:, :most] + 0.7 * torch.randn(n, most, v, generator=g, device="cuda")).reshape(
        n * most, v)
    noise = torch.rand(n * most, v, generator=g, device="cuda").clamp_(1e-20, 1 - 6e-8).log().neg().log().neg()
    tokens = ((near + noise) if has_draft else near).argmax(1) if most else torch.zeros(0, device="cuda")
    draft = None
    if has_draft and most:
        draft = rows(g, n * most, v, x, pad, off)
        draft.copy_(near)
    if form == "probs":
        target.copy_(torch.softmax(target.float(), 1))
        if draft is not None:
            draft.copy_(torch.softmax(draft.float(), 1))
    n_draft = torch.full((n,), most, dtype=torch.int32, device="cuda")
    n_draft[1::3] = most // 2
    u = torch.rand(n, most + 1, generator=g, device="cuda")
    return target, draft, tokens.int().view(n, most), n_draft, u


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["logits", "probs"])
@pytest.mark.parametrize("has_draft", [True, False])
@pytest.mark.parametrize("v", [1, 2, 63, 1024, 1025, 9001])
def test_types_and_sizes(x, form, has_draft, v):
    check(*case(7, 3, v, x, form, has_draft, seed=v), form=form)


@pytest.mark.parametrize("n,most,v", [(1, 0, 5000), (3, 0, 300), (1, 1, 32001), (1, 4, 151936), (2, 15, 4097), (33, 5, 700),
                                      (300, 2, 150), (4, 2, 300000)])
def test_shapes(n, most, v):
    check(*case(n, most, v, seed=n))
    check(*case(n, most, v, "bf16", has_draft=False, seed=n + 1))


@pytest.mark.parametrize("v", [300000, 1300001])
def test_large_vocabularies(v):
    """More parts of a row than lanes, and more tiles than threads hold, greedy and not."""
    import torch
    target, draft, tokens, n_draft, u = case(3, 1, v, seed=v)
    n_draft.fill_(1)
    temp = torch.tensor([0.0, 0.8, 0.0], device="cuda")
    tokens[0] = target.view(3, 2, v)[0, 0].argmax().int()
    check(target, draft, tokens, n_draft, u, temp=temp)
    check(target, None, tokens, n_draft, u, temp=temp)
    check(torch.softmax(target, 1), torch.softmax(draft, 1), tokens, n_draft, u, form="probs")


def test_many_passes_a_chunk():
    """Enough rows that a workgroup takes several passes over its part of a row."""
    target, draft, tokens, n_draft, u = case(48, 7, 40000, "f32", seed=5)
    check(target, draft, tokens, n_draft, u)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("pad,off", [(1, 0), (0, 1), (5, 3), (8, 8)])
def test_rows_of_any_alignment(x, pad, off):
    check(*case(5, 3, 5003, x, seed=pad, pad=pad, off=off))


@pytest.mark.parametrize("has_draft", [True, False])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_temperatures(has_draft, x):
    import torch
    target, draft, tokens, n_draft, u = case(24, 3, 3001, x, has_draft=has_draft, seed=9)
    temp = torch.tensor([0.0, 1.0, 0.7, 1.5, 0.01, 100.0, 0.0, float("inf")] * 3, device="cuda")
    # greedy drafts that are right, and the target's own tie of two largest
    best = target.float().argmax(1).view(24, 4)
    tokens[0] = best[0, :3].int()
    target[6 * 4, 17] = target[6 * 4, 2500] = 30.0
    tokens[6, 0] = 17
    target[8 * 4, 17] = target[8 * 4, 2500] = 30.0
    temp[8] = 0.0
    tokens[8, 0] = 2500                       # not the lowest of the two
    temp[7::8] = 3.0
    out, acc = check(target, draft, tokens, n_draft, u, temp=temp)
    assert acc[0] == 3 and acc[6] >= 1 and acc[8] == 0 and out[8, 0] == 17
    temp[7] = float("inf")                    # every token that is not masked alike
    target[7 * 4: 8 * 4, 100:] = -float("inf")
    out, _ = B.q2_0_draft_verify(target, None, tokens, n_draft, u, temperature=temp)
    assert int(out[7].max()) < 3001
    temp[3], temp[4] = -1.0, float("nan")
    check(target, draft, tokens, n_draft, u, temp=torch.where(torch.isinf(temp), 1.0, temp))


@pytest.mark.parametrize("size,t", [(1.0, 1e-3), (1.0, 1e-6), (1.0, 1e-8), (1.0, 1e-10), (1.0, 1e-20), (1.0, 1e-30), (1e6, 1.0),
                                    (1e6, 1e-4), (1e9, 300.0), (1e30, 1.0), (1e30, 1e27), (1e38, 1e37), (1e-30, 1e-30), (1e20, 1e25),
                                    (1e-20, 1.0)])
def test_logits_and_temperatures_out_of_proportion(size, t):
    """Rows whose largest values are a few float32 steps apart, the others anywhere, masks among them; a temperature of the
    size of a step tells the largest apart, others not."""
    import torch
    n, v = 24, 3000
    g = torch.Generator(device="cuda").manual_seed(21)
    target = size * torch.randn(n, v, generator=g, device="cuda")
    target[:, ::7] = -float("inf")
    top = torch.full((n,), min(5.3 * size, 3e38), device="cuda")      # (float32 ends at 3.4e38)
    for i in range(40):
        target[:, 50 * i + 1] = top
        if i % 3 == 0:
            top = torch.nextafter(top, torch.zeros_like(top))
    target[1::2, 2:] = -target[1::2, 2:].abs()       # negative ones, the largest at the front
    target[1::2, 7::7] = -float("inf")
    u = torch.rand(n, 1, generator=g, device="cuda")
    temp = torch.full((n,), t, device="cuda")
    none = torch.zeros(n, 0, dtype=torch.int32, device="cuda")
    check(target, None, none, torch.zeros(n, dtype=torch.int32, device="cuda"), u, temp=temp)
    tokens = torch.full((n // 2, 1), 1, dtype=torch.int32, device="cuda")
    draft = target[::2].roll(1, 0).contiguous()
    check(target, draft, tokens, torch.ones(n // 2, dtype=torch.int32, device="cuda"), u.view(n // 2, 2), temp=temp[: n // 2])


def test_draft_counts_and_tokens():
    import torch
    target, draft, tokens, n_draft, u = case(9, 4, 600, seed=11)
    n_draft.copy_(torch.tensor([0, 1, 2, 3, 4, -1, 5, 2 ** 31 - 1, -(2 ** 31)]))
    for d in (draft, None):
        out, acc = check(target, d, tokens, n_draft, u)
        assert torch.all(out[5:] == -1) and torch.all(acc[5:] == 0)
    tokens[1, 0], tokens[2, 1], tokens[3, 0], tokens[4, 3] = -1, 600, 2 ** 31 - 1, -5
    n_draft[1:5] = 4
    for d in (draft, None):
        check(target, d, tokens, n_draft, u)
    check(torch.softmax(target, 1), torch.softmax(draft, 1), tokens, n_draft, u, form="probs")


def test_masked_tokens_and_bad_rows():
    import torch
    inf, nan = float("inf"), float("nan")
    for has_draft in (True, False):
        target, draft, tokens, n_draft, u = case(16, 2, 2100, has_draft=has_draft, seed=13)
        n_draft.fill_(2)
        t = target.view(16, 3, 2100)
        t[0, :, 7:] = -inf                    # seven tokens left
        t[1, 0, :] = -inf                     # none
        t[2, 1, :] = -inf
        t[3, 2, :] = -inf
        t[4, 0, 2099] = nan
        t[5, 1, 0] = nan
        t[6, 2, 1024] = nan
        t[7, 0, 5] = inf
        t[8, 2, 2000] = inf
        t[9, :, :-1] = -inf                   # the last token alone
        t[10, :, 1:] = -inf                   # the first
        t[11, :, :2000] = -inf                # whole tiles of nothing before
        tokens[11] = 2050
        if has_draft:
            d = draft.view(16, 2, 2100)
            d[12, 0, :] = -inf
            d[13, 1, 3] = nan
            d[14, 0, 3] = inf
            d[15, 0, ::2] = -inf
        temp = torch.ones(16, device="cuda")
        check(target, draft, tokens, n_draft, u)
        check(target, draft, tokens, n_draft, u, temp=temp)
        temp[::2] = 0.0
        check(target, draft, tokens, n_draft, u, temp=temp)
    # what is never needed may hold anything
    target, draft, tokens, n_draft, u = case(4, 3, 800, seed=14)
    n_draft.copy_(torch.tensor([1, 1, -1, 1]))
    target.view(4, 4, 800)[:, 2:] = nan
    draft.view(4, 3, 800)[:, 1:] = nan
    out, _ = check(target, draft, tokens, n_draft, u)
    assert torch.all(out[[0, 1, 3], 0] >= 0)


def test_numbers_at_the_ends():
    import torch
    for form in ("logits", "probs"):
        target, draft, tokens, n_draft, u = case(6, 2, 1500, form=form, seed=15)
        below = float(np.nextafter(np.float32(1), np.float32(0)))
        for value in (0.0, below, 1.0):
            u.fill_(value)
            check(target, draft, tokens, n_draft, u, form=form)
            check(target, None, tokens, n_draft, u, form=form)


def test_one_distribution_takes_every_draft():
    import torch
    target, _, _, n_draft, u = case(8, 5, 900, seed=16)
    n_draft.fill_(5)
    draft = target.view(8, 6, 900)[:, :5].reshape(40, 900).contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.multinomial(torch.softmax(draft, 1), 1, generator=g).int().view(8, 5)
    _, acc = check(target, draft, tokens, n_draft, u)
    assert torch.all(acc == 5)


def test_nothing_left_of_the_difference():
    """Probabilities of which the draft's are nowhere below: the token comes from the target's."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(17)
    q = torch.softmax(torch.randn(4, 3000, generator=g, device="cuda"), 1)
    p = torch.cat([0.25 * q, q], 1).view(8, 3000)
    tokens = torch.randint(0, 3000, (4, 1), generator=g, device="cuda", dtype=torch.int32)
    u = torch.tensor([[0.9, 0.1], [0.9, 0.999], [0.5, 0.0], [0.1, 0.5]], device="cuda")
    _, acc = check(p, q, tokens, torch.ones(4, dtype=torch.int32, device="cuda"), u, form="probs")
    assert acc.tolist() == [0, 0, 0, 1]
    # negative values count as nothing where a token is drawn, and rows of nothing give -1
    p[0, ::2] = -1.0
    p[2] = 0.0
    p[4] = -2.0
    out, _ = check(p, q, tokens, torch.ones(4, dtype=torch.int32, device="cuda"), u, form="probs")
    assert out[1, 0] == out[2, 0] == -1


def test_how_often_tokens_come():
    """One draft of a five-token language, 40000 sequences: the token that comes first is distributed as the target has it."""
    import torch
    n = 40000
    p = torch.tensor([0.5, 0.2, 0.15, 0.1, 0.05], device="cuda")
    q = torch.tensor([0.1, 0.3, 0.2, 0.2, 0.2], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(18)
    tokens = torch.multinomial(q.expand(n, 5), 1, generator=g).int()
    u = torch.rand(n, 2, generator=g, device="cuda")
    nd = torch.ones(n, dtype=torch.int32, device="cuda")
    out, acc = B.q2_0_draft_verify(p.log().expand(2 * n, 5).contiguous(), q.log().expand(n, 5).contiguous(), tokens, nd, u)
    torch.cuda.synchronize()
    share = torch.bincount(out[:, 0].long(), minlength=5).double() / n
    # five standard deviations of a share of 40000 draws
    assert torch.all((share - p.double()).abs() < 5 * (p.double() * (1 - p.double()) / n).sqrt())
    assert abs(acc.double().mean().item() - torch.minimum(p, q).sum().item()) < 5 * (0.25 / n) ** 0.5


def test_rows_past_32_bit_offsets():
    import torch
    v, n = 151936, 14300                      # 2.17e9 elements of target, 4.3 GB
    target = torch.empty(n, v, dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(19)
    target[:] = rows(g, 1, v, "f16")
    at = torch.arange(n, device="cuda") * 10 % v
    target[torch.arange(n, device="cuda"), at] = 60.0          # all but e^-30 of the whole
    u = torch.rand(n, 1, generator=g, device="cuda").clamp_(0.001, 0.999)
    out, acc = B.q2_0_draft_verify(target, None, torch.zeros(n, 0, dtype=torch.int32, device="cuda"),
                                   torch.zeros(n, dtype=torch.int32, device="cuda"), u)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 0].long(), at) and torch.all(acc == 0)


def test_same_every_time_and_workspace_of_any_content():
    import torch
    target, draft, tokens, n_draft, u = case(20, 4, 20000, seed=20)
    need = B.draft_verify_workspace_bytes(20, 4, 20000, B.Q2_0_ACT_F32, 0, 1)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got = check(target, draft, tokens, n_draft, u, workspace=ws)
        first = first or got
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t", [1.0, 0.25])
def test_where_probabilities_end(x, t):
    """Next to nothing is still taken where the draft gave it less; below 2^-1000 of the largest it is nothing."""
    import torch
    ends = {"f32": 690.0, "f16": 690.0, "bf16": 688.0}[x], {"f32": 697.0, "f16": 697.0, "bf16": 700.0}[x]
    target = torch.zeros(4, 70, device="cuda", dtype=types()[x])    # (two sequences' rows; 1000 ln 2 = 693.1)
    target[0, 9], target[2, 9] = -ends[0] * t, -ends[1] * t
    draft = torch.zeros(2, 70, device="cuda", dtype=types()[x])
    draft[:, 9] = -float("inf")
    tokens = torch.full((2, 1), 9, dtype=torch.int32, device="cuda")
    u = torch.full((2, 2), 0.5, device="cuda")
    _, acc = B.q2_0_draft_verify(target, draft, tokens, torch.ones(2, dtype=torch.int32, device="cuda"), u,
                                 form=FORM["logits"], temperature=torch.full((2,), t, device="cuda"))
    assert acc.tolist() == [1, 0]


def border(sign):
    """(temperature, x, y): neighbouring float32 values with x > y on either side of |value log2(e) / temperature| = 2^28, where
    sums change their reference, and the value inside it some 0.45 from a whole number there.  y counts about 2^-16 of x."""
    for i in range(100000):
        t = np.float32(1e-8) * (np.float32(1) + np.float32(i) * np.float32(2.0 ** -20))
        k = 1.4426950408889634 / float(t)
        inside = np.float32(2.0 ** 28 / k)
        while abs(float(inside)) * k >= 2.0 ** 28:
            inside = np.nextafter(inside, np.float32(0))
        while abs(float(np.nextafter(inside, np.float32(9)))) * k < 2.0 ** 28:
            inside = np.nextafter(inside, np.float32(9))
        outside = np.nextafter(inside, np.float32(9))
        off = float(inside) * k - np.rint(float(inside) * k)
        if 0.4 < abs(off) < 0.5 and (float(outside) - float(inside)) * k < 20:
            return (float(t), float(outside), float(inside), off) if sign > 0 else (float(t), -float(inside), -float(outside), -off)
    raise AssertionError("no such values")


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("where", ["threads", "chunks", "passes", "many chunks"])
def test_values_on_either_side_of_a_references_border(sign, where):
    """The largest logit and its lower neighbours in one pass, in other chunks of the row, in two passes of a thread, and in two
    chunks that one lane joins; the number that decides lies halfway between the probability and what it would be with one
    side's reference for both."""
    import torch
    t, high, low, off = border(sign)
    v, n, most, at = {"threads": (4096, 3, 1, 7), "chunks": (100000, 3, 1, 7), "passes": (40000, 76, 7, 4096),
                      "many chunks": (300000, 3, 1, 4100)}[where]
    row = torch.full((v,), low, dtype=torch.float32)
    if where == "passes":                     # of 4096 values: 16 of a thread in the first, its next in the second
        row[:] = -float("inf")
        row[(torch.arange(4)[:, None] * 1024 + torch.arange(4)).flatten()] = low
    if where == "many chunks":
        row[: 65 * 4096] = -float("inf")
    row[at] = high
    others = int((row == low).sum()) * 2.0 ** (-(high - low) / t * 1.4426950408889634)
    p = 1 / (1 + others)
    # the sum of the part whose reference is a whole number, taken as if it were about its largest value
    wrong = 1 / (1 + others * 2.0 ** off) if sign > 0 else 1 / (1 + others * 2.0 ** -off)
    u = np.float32((p + wrong) / 2)
    assert min(p, wrong) < float(u) < max(p, wrong)
    target = row.cuda().expand(n * (most + 1), v).contiguous()
    tokens = torch.full((n, most), at, dtype=torch.int32, device="cuda")
    uu = torch.full((n, most + 1), float(u), device="cuda")
    check(target, None, tokens, torch.full((n,), most, dtype=torch.int32, device="cuda"), uu, temp=torch.full((n,), t, device="cuda"))


def test_choices_that_float32_does_not_decide():
    """Two-token rows whose probability lies next to the number that decides, closer than a float32 step by some 10^5.  An
    exponential is within 2^-45 of itself and a probability, a quotient of two by their sum, within 2^-44 and a few roundings
    of 2^-53: what is further off than 2^-43 has to be decided as the definition says."""
    import torch
    x = np.random.default_rng(31).uniform(-8, 8, 6000000).astype(np.float32)
    p = 1 / (1 + np.exp(-x.astype(np.longdouble)))
    u = p.astype(np.float32)
    off = np.abs(p / u.astype(np.longdouble) - 1)
    some = np.nonzero((off > 2.0 ** -43) & (off < 2.0 ** -40))[0]
    n = len(some)
    assert n > 50
    target = torch.zeros(n, 2, 2, device="cuda")
    target[:, 0, 1] = torch.from_numpy(x[some]).cuda()
    tokens, n_draft = torch.ones(n, 1, dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda")
    uu = torch.from_numpy(u[some]).cuda()[:, None].repeat(1, 2)
    _, acc = B.q2_0_draft_verify(target.view(2 * n, 2), None, tokens, n_draft, uu)
    assert np.array_equal(acc.cpu().numpy() == 1, u[some] < p[some])


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("side", ["target", "draft"])
def test_given_probabilities_of_a_drafted_token(x, value, side):
    """A drafted token with a value that is none is not taken, whatever its number; of a target like that nothing follows."""
    import torch
    target, draft, tokens, n_draft, u = case(6, 3, 700, x, "probs", seed=41)
    n_draft.fill_(3)
    draft.copy_(target.reshape(6, 4, 700)[:, :3].reshape(18, 700))       # (each draft is taken where u < 1)
    tokens.copy_(draft.argmax(1).int().view(6, 3))
    for s in range(6):
        rows, per = (target, 4) if side == "target" else (draft, 3)
        rows[s * per + s % 3, int(tokens[s, s % 3])] = float(value)
    u[3:] = 0.0
    out, acc = B.q2_0_draft_verify(target, draft, tokens, n_draft, u, form=FORM["probs"])
    assert acc.tolist() == [0, 1, 2, 0, 1, 2]
    for s in range(6):
        assert out[s, : s % 3].tolist() == tokens[s, : s % 3].tolist()
        assert side == "draft" or torch.all(out[s, s % 3:] == -1)
    if side == "target":
        out, acc = B.q2_0_draft_verify(target, None, tokens, n_draft, torch.zeros_like(u), form=FORM["probs"])
        assert acc.tolist() == [0, 1, 2, 0, 1, 2] and all(out[s, s % 3] == -1 for s in range(6))


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("v", [3, 1000, 20011])
def test_given_probabilities_below_zero(x, v):
    """They count as 0, the draft's too: such rows give what the same rows with zeros in those places do."""
    import torch
    n = 40
    target, draft, tokens, n_draft, u = case(n, 3, v, x, "probs", seed=v)
    g = torch.Generator(device="cuda").manual_seed(v)
    for rows in (target, draft):
        rows[torch.rand(rows.shape, generator=g, device="cuda") < 0.4] = 0.0
    draft[:, v - 1] = 0.25                                      # (no draft of nothing)
    keep = [r.clone() for r in (target, draft)]
    tokens[::4] = torch.randint(0, v, tokens[::4].shape, generator=g, device="cuda", dtype=torch.int32)
    want = check(target, draft, tokens, n_draft, u, form="probs")
    for rows in (target, draft):
        rows[rows == 0] = -0.75
        rows[1::3][rows[1::3] < 0] = -float("inf")
    out, acc = B.q2_0_draft_verify(target, draft, tokens, n_draft, u, form=FORM["probs"])
    assert torch.equal(acc, want[1]) and torch.equal(out, want[0])
    # a token of no probability is not taken because the draft's is below 0
    target, draft = keep
    target[:, 0], draft[:, 0] = 0.0, -0.5
    tokens.zero_()
    n_draft.fill_(3)
    _, acc = B.q2_0_draft_verify(target, draft, tokens, n_draft, u, form=FORM["probs"])
    assert torch.all(acc == 0)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("v", [5, 513, 9001])
def test_given_probabilities_of_the_deciding_rows(x, v):
    """NaN or +inf anywhere in the rows of the place that decides, and rows with nothing above 0: no token follows."""
    import torch
    nan, inf = float("nan"), float("inf")
    n = 12
    target, draft, tokens, n_draft, u = case(n, 2, v, x, "probs", seed=v)
    t, d = target.view(n, 3, v), draft.view(n, 2, v)
    n_draft.fill_(2)
    tokens.fill_(v - 1)
    t[:, :, v - 1], d[:, :, v - 1] = 0.0, 0.5                   # refused at once
    t[0, 0, 1], t[1, 0, v - 2], t[2, 0, 2] = nan, inf, -inf    # (-inf: below 0, nothing)
    d[3, 0, 1], d[4, 0, v - 2] = nan, inf
    t[6, 0] = 0.0
    d[7, 0] = 0.0
    d[8, 0], tokens[8, 0] = 0.0, v                              # a token that is none, and a draft of nothing
    d[9, 0] = -0.25
    t[10, 0, v - 1] = nan
    t[11, 0, v - 2], d[11, 0, v - 2] = inf, inf
    out, acc = B.q2_0_draft_verify(target, draft, tokens, n_draft, u, form=FORM["probs"])
    assert torch.all(acc == 0) and torch.all(out[:, 1:] == -1)
    assert [int(o) >= 0 for o in out[:, 0]] == [s in (2, 5) for s in range(n)], out[:, 0]
    # found drafts: the token itself has what is none
    t[:, :, v - 1] = 0.0
    t[0, 0, v - 1], t[1, 0, v - 1], t[2, 0, v - 1], tokens[2, 0] = nan, inf, nan, -1
    t[3:] = torch.softmax(torch.randn(n - 3, 3, v, device="cuda"), 2).to(t.dtype)
    out, acc = B.q2_0_draft_verify(target, None, tokens, n_draft, torch.full_like(u, 0.9999), form=FORM["probs"])
    assert out[:3, 0].tolist() == [-1, -1, -1] and torch.all(acc[:3] == 0) and torch.all(out[3:, 0] >= 0)
    # rows of places that were passed are not looked through, but for the drafted token's values
    target, draft, tokens, n_draft, u = case(2, 1, v, x, "probs", seed=v)
    n_draft.fill_(1)
    draft.copy_(target.view(2, 2, v)[:, 0])
    tokens.copy_(draft.argmax(1).int()[:, None])
    target[0, (int(tokens[0]) + 1) % v], draft[1, (int(tokens[1]) + 1) % v] = nan, inf
    _, acc = B.q2_0_draft_verify(target, draft, tokens, n_draft, u, form=FORM["probs"])
    assert acc.tolist() == [1, 1]


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_infinite_temperatures(x):
    """Every token that is not masked alike, up to the documented end of temperatures."""
    import torch
    target, draft, tokens, n_draft, u = case(12, 2, 3001, x, seed=43)
    target.view(12, 3, 3001)[:, :, 100:] = -float("inf")
    draft.view(12, 2, 3001)[::2, :, 50:] = -float("inf")
    tokens.remainder_(120)
    temp = torch.full((12,), float("inf"), device="cuda")
    temp[::3] = 1e30
    for d in (draft, None):
        out, _ = check(target, d, tokens, n_draft, u, temp=temp)
        assert int(out.max()) < 100
    u[:, 2] = (torch.arange(12, device="cuda") * 8 + 0.5) / 100
    out, _ = check(target, None, tokens, torch.zeros_like(n_draft), u, temp=temp)
    assert out[:, 0].tolist() == [8 * s for s in range(12)]
