"""Position rotation and paged cache append against the definition in 64 bits, on every
alignment, type, style and partial rotation, with padding, bad pages and bad positions."""

import numpy as np
import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

# A turned element: two products and a sum in f32 (3 roundings of at most |a c| + |b s|), then
# one rounding to the cache's type (unit roundoff u; below the half's normal range 2^-25).
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
STYLE = {"half": B.Q2_0_ROPE_HALF, "pairs": B.Q2_0_ROPE_PAIRS}


def types():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def turned(x, table, pos, rot, style):
    """x (tokens, heads, dim) float64 -> (result, |a c| + |b s|)."""
    half = rot // 2
    i = np.arange(half)
    ia, ib = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
    out, size = x.copy(), np.zeros_like(x)
    c, s = table[pos][:, None, :half], table[pos][:, None, half:]
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia], size[..., ib] = abs(a * c) + abs(b * s), abs(b * c) + abs(a * s)
    return out, size


def close(got, ref, size, u, what):
    got = got.double().cpu().numpy()
    err = np.abs(got - ref)
    tol = u * np.abs(ref) + 3 * 2.0 ** -24 * (1 + u) * size + 2.0 ** -25
    assert np.all(err <= tol), "%s: worst %.3g of its tolerance" % (what, np.max(err / tol))


def run(tokens, n_q, n_kv, dim, rot, style, xt, ct, page, layout="pages", off=0, pad=0, seed=0, n_seqs=3):
    import torch
    ty = types()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = np.array([tokens // n_seqs + (1 if i < tokens % n_seqs else 0) for i in range(n_seqs)])
    start = np.array([0, 5, 3 * page + 1])[:n_seqs]
    seq = np.repeat(np.arange(n_seqs), lens).astype(np.int32)
    pos = np.concatenate([s + np.arange(n) for s, n in zip(start, lens)]).astype(np.int32)
    cols = int((start + lens).max() + page - 1) // page
    n_pages = n_seqs * cols + 2
    table = rng.permutation(n_pages)[: n_seqs * cols].reshape(n_seqs, cols).astype(np.int32)
    shape = (n_pages, n_kv, page, dim) if layout == "pages" else (n_pages, page, n_kv, dim)
    kc, vc = (torch.randn(shape, generator=g, device="cuda").to(ty[ct]) for _ in range(2))
    if layout != "pages":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    k0, v0 = kc.double().cpu().numpy(), vc.double().cpu().numpy()

    def src(heads):
        buf = torch.randn(tokens * (heads * dim + pad) + off, generator=g, device="cuda").to(ty[xt])
        return buf[off:].view(tokens, heads * dim + pad)[:, : heads * dim]

    q, k, v = src(n_q), src(n_kv), src(n_kv)
    if style == "none":
        rope, rot = None, 0
    else:
        ang = rng.uniform(-4, 4, size=(int(pos.max()) + 1, rot // 2))
        rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    q_out = torch.full((tokens, n_q * dim + 8), float("inf"), device="cuda").to(ty[ct])
    got = B.q2_0_kv_append(kc, vc, torch.from_numpy(table).cuda(), torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                           k, v, rope=rope, style=STYLE.get(style, 0), q=q, q_out=q_out[:, : n_q * dim])
    torch.cuda.synchronize()
    assert torch.isinf(q_out[:, n_q * dim:]).all(), "wrote past a q row"
    tab = np.zeros((1, 0)) if rope is None else rope.double().cpu().numpy()
    hq, hk, hv = (t.double().cpu().numpy().reshape(tokens, -1, dim) for t in (q, k, v))
    p = pos if rope is not None else np.zeros_like(pos)
    rq, sq = turned(hq, tab, p, rot, "half" if style == "none" else style)
    rk, sk = turned(hk, tab, p, rot, "half" if style == "none" else style)
    close(got, rq.reshape(tokens, -1), sq.reshape(tokens, -1), U[ct], "q")
    where, row = table[seq, pos // page], pos % page
    sk0 = np.zeros_like(k0)
    k0[where, :, row], sk0[where, :, row] = rk, sk
    # rows that were not appended keep their bits; v is only rounded (exact where the type is the same)
    kk = kc.double().cpu().numpy()
    kept = np.ones(kk.shape[:1] + kk.shape[2:3], bool)
    kept[where, row] = False
    assert np.array_equal(kk.transpose(0, 2, 1, 3)[kept], k0.transpose(0, 2, 1, 3)[kept])
    close(kc, k0, sk0, U[ct], "k")
    v0[where, :, row] = v.to(ty[ct]).double().cpu().numpy().reshape(tokens, n_kv, dim)
    assert np.array_equal(vc.double().cpu().numpy(), v0), "v"


@pytest.mark.parametrize("ct", ["f16", "bf16"])
@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("style", ["half", "pairs", "none"])
def test_types_dims_styles(ct, xt, dim, style):
    run(37, 6, 2, dim, dim, style, xt, ct, 16, seed=dim)


@pytest.mark.parametrize("rot", [2, 8, 20, 24, 64, 126, 128])
@pytest.mark.parametrize("style", ["half", "pairs"])
def test_partial_rotation(rot, style):
    run(11, 3, 1, 128, rot, style, "f32", "bf16", 7, seed=rot)


@pytest.mark.parametrize("tokens,n_seqs", [(1, 1), (2, 2), (3, 3), (64, 1), (1001, 3)])
def test_token_counts(tokens, n_seqs):
    run(tokens, 32, 8, 128, 128, "half", "f32", "bf16", 64, seed=tokens, n_seqs=n_seqs)


@pytest.mark.parametrize("xt", ["f32", "f16"])
@pytest.mark.parametrize("off,pad", [(1, 0), (0, 1), (4, 4), (3, 5)])
def test_unaligned_rows(xt, off, pad):
    run(9, 4, 2, 64, 64, "half", xt, "f16", 16, off=off, pad=pad, seed=off)


@pytest.mark.parametrize("page", [1, 3, 16, 1000])
@pytest.mark.parametrize("layout", ["pages", "tokens"])
def test_pages_and_layouts(page, layout):
    run(50, 4, 4, 64, 32, "pairs", "bf16", "bf16", page, layout=layout, seed=page)


def test_without_q():
    import torch
    kc = torch.zeros(4, 1, 16, 64, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = torch.ones(2, 64, device="cuda"), torch.full((2, 64), 2.0, device="cuda")
    assert B.q2_0_kv_append(kc, vc, i(3, 1).view(1, 2), i(0, 0), i(0, 17), k, v) is None
    torch.cuda.synchronize()
    assert (kc[3, 0, 0] == 1).all() and (kc[1, 0, 1] == 1).all() and kc.sum() == 128
    assert (vc[3, 0, 0] == 2).all() and (vc[1, 0, 1] == 2).all() and vc.sum() == 256


def test_tokens_that_are_not_stored():
    """Padding (seq -1), sequences, positions and pages that do not exist: nothing is stored,
    the q row is written, and turned by NaN where the position is outside the table."""
    import torch
    kc = torch.zeros(4, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i(2, -1, 4, 1).view(1, 4)
    seq = i(-1, 1, 0, 0, 0, 0, 0)
    pos = i(0, 0, -3, 4, 8, 16, 12)      # padding, no such sequence, negative, page -1, page 4, past the table, stored
    n = seq.numel()
    k = torch.ones(n, 128, device="cuda")
    q = torch.ones(n, 128, device="cuda")
    rope = torch.cat([torch.ones(14, 16), torch.zeros(14, 16)], 1).cuda()      # positions 0 .. 13: no turn
    out = B.q2_0_kv_append(kc, vc, table, seq, pos, k, k, rope=rope, q=q)
    torch.cuda.synchronize()
    want = torch.zeros_like(kc)
    want[1, :, 0] = 1
    assert torch.equal(kc, want) and torch.equal(vc, want)
    o = out.view(n, 2, 64)
    for t, p in enumerate(pos.tolist()):
        assert (o[t, :, 32:] == 1).all()
        assert torch.isnan(o[t, :, :32]).all() if p < 0 or p >= 14 else (o[t, :, :32] == 1).all(), t


def test_position_past_the_table_is_stored_as_nan():
    import torch
    kc = torch.zeros(1, 1, 4, 64, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rope = torch.ones(2, 64, device="cuda")
    one = torch.ones(1, 64, device="cuda")
    B.q2_0_kv_append(kc, vc, i(0).view(1, 1), i(0), i(3), one, one, rope=rope)
    torch.cuda.synchronize()
    assert torch.isnan(kc[0, 0, 3]).all() and (vc[0, 0, 3] == 1).all() and kc[0, 0, :3].abs().sum() == 0


def test_refusals():
    import torch
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t, s, p = i(0, 1).view(1, 2), i(0), i(0)
    k = torch.zeros(1, 128, device="cuda")
    with pytest.raises(ValueError):
        B.q2_0_kv_append(kc.float(), kc.float(), t, s, p, k, k)
    with pytest.raises(ValueError):
        B.q2_0_kv_append(kc, kc[:3], t, s, p, k, k)
    with pytest.raises(ValueError):
        B.q2_0_kv_append(kc, kc, t, s.long(), p, k, k)
    with pytest.raises(ValueError):
        B.q2_0_kv_append(kc, kc, t, s, p, k, k.half())
    with pytest.raises(ValueError):
        B.q2_0_kv_append(kc, kc, t, s, p, k, k[:, :100])
    with pytest.raises(ValueError):
        B.q2_0_kv_append(kc, kc, t, s, p, k, k, q=torch.zeros(1, 100, device="cuda"))
    with pytest.raises(B.Q2_0Error):
        B.q2_0_kv_append(kc, kc.clone(), t, s, p, k, k, rope=torch.zeros(4, 7, device="cuda"))
    with pytest.raises(B.Q2_0Error):
        B.q2_0_kv_append(kc, kc.clone(), t, s, p, k, k, style=5)
