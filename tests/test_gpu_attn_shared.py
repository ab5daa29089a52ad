"""Shared-prefix attention over the paged cache against the definition in 64 bits: types, head
layouts, lengths from none to long, page sizes that end inside a key tile, causal draft
tokens, and places that no query sees holding NaN."""

import numpy as np
import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

# o = sum p v / sum p.  The softmax weights are rounded to the cache's type (u each), the scores err by
# (dim + 4) f32 roundings of scale * sum |q k| (dim products and sums, scale, exponential), which a weight
# takes as a relative error, in the sum and below the line; the result is rounded once (u).
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def make(seed, n_seqs, n_qt, n_q, n_kv, dim, ct, page, prefix, own, layout="pages", hole=float("nan"), spread=1.5):
    """Inputs on the GPU; every cache row that no sequence holds is `hole`."""
    import torch
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[ct]
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = np.array([prefix + n for n in own], dtype=np.int32)
    cols = max(1, int(max(lens.max(), prefix) + page - 1) // page)
    shared = prefix // page
    n_pages = shared + n_seqs * (cols - shared) + 1
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.empty((n_seqs, cols), np.int32)
    table[:, :shared] = perm[:shared]
    table[:, shared:] = perm[shared : shared + n_seqs * (cols - shared)].reshape(n_seqs, -1)
    shape = (n_pages, n_kv, page, dim) if layout == "pages" else (n_pages, page, n_kv, dim)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
    if layout != "pages":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if prefix % page:
        edge = table[:, shared]
        for t in (k, v):
            t[edge.tolist(), :, : prefix % page] = t[int(edge[0]), :, : prefix % page].clone()
    held = np.zeros((n_pages, page), bool)
    for s in range(n_seqs):
        i = np.arange(max(prefix, lens[s]))
        held[table[s][i // page], i % page] = True
    hole_at = torch.from_numpy(~held).cuda()
    for t in (k, v):
        t.transpose(1, 2)[hole_at] = hole
    q = (spread * torch.randn(n_seqs * n_qt, n_q * dim, generator=g, device="cuda")).to(dt)
    return q, k, v, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()


def reference(q, k, v, table, lens, scale, n_qt, u):
    """(result, tolerance) in float64 from the definition, row by row."""
    kc, vc = k.double().cpu().numpy(), v.double().cpu().numpy()
    _, n_kv, page, dim = kc.shape
    rows = q.double().cpu().numpy().reshape(q.shape[0], n_kv, -1, dim)
    tab = table.cpu().numpy()
    out, tol = np.zeros(rows.shape), np.zeros(rows.shape)
    for s, length in enumerate(lens.tolist()):
        for j in range(n_qt):
            n = length - n_qt + 1 + j
            if n <= 0:
                continue
            i = np.arange(n)
            ks = kc[tab[s][i // page], :, i % page].transpose(1, 0, 2)       # (n_kv, n, dim)
            vs = vc[tab[s][i // page], :, i % page].transpose(1, 0, 2)
            x = rows[s * n_qt + j]
            sc = scale * (x @ ks.transpose(0, 2, 1))
            size = scale * (np.abs(x) @ np.abs(ks).transpose(0, 2, 1)).max(axis=2, keepdims=True)
            p = np.exp(sc - sc.max(axis=2, keepdims=True))
            p /= p.sum(axis=2, keepdims=True)
            o = p @ vs
            a = p @ np.abs(vs)
            delta = (dim + 4) * 2.0 ** -24 * size + n * 2.0 ** -24
            out[s * n_qt + j] = o
            tol[s * n_qt + j] = (u + 2 * delta) * a + u * np.abs(o) + 2.0 ** -24
    return out.reshape(q.shape), tol.reshape(q.shape)


def check(got, ref, tol, what=""):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(np.isfinite(err)), what + ": not finite"
    assert np.all(err <= tol), "%s: worst %.3g of its tolerance" % (what, np.max(err / tol))


def run(seed, n_seqs, n_qt, n_q, n_kv, dim, ct, page, prefix, own, layout="pages", max_len=None, **kw):
    import torch
    q, k, v, table, lens = make(seed, n_seqs, n_qt, n_q, n_kv, dim, ct, page, prefix, own, layout, **kw)
    scale = dim ** -0.5
    out = torch.full((q.shape[0], q.shape[1] + 8), float("inf"), device="cuda").to(q.dtype)
    need = B.attn_shared_workspace_bytes(n_seqs, n_q, n_kv, dim, n_qt, prefix, max_len or table.shape[1] * page)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")          # partials hold nothing beforehand
    got = B.q2_0_attn_shared(q, k, v, table, lens, scale, prefix_len=prefix, n_qt=n_qt, max_len=max_len,
                             out=out[:, : q.shape[1]], workspace=ws)
    torch.cuda.synchronize()
    assert torch.isinf(out[:, q.shape[1]:]).all(), "wrote past a row"
    ref, tol = reference(q, k, v, table, lens, scale, n_qt, U[ct])
    check(got, ref, tol, "prefix %d own %s" % (prefix, list(own)[:4]))
    again = B.q2_0_attn_shared(q, k, v, table, lens, scale, prefix_len=prefix, n_qt=n_qt, max_len=max_len)
    assert torch.equal(again, got), "two runs differ"
    return q, k, v, table, lens, got


@pytest.mark.parametrize("ct", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n_q,n_kv", [(1, 1), (8, 1), (14, 2), (32, 8), (24, 1)])
def test_types_and_heads(ct, dim, n_q, n_kv):
    run(1, 3, 1, n_q, n_kv, dim, ct, 16, 70, [1, 40, 133])


@pytest.mark.parametrize("own", [[1], [2], [15], [16], [17], [31], [32], [33], [64], [127], [128], [129], [777], [5000]])
def test_one_sequence_lengths(own):
    run(2, 1, 1, 8, 2, 128, "bf16", 16, 0, own)


@pytest.mark.parametrize("prefix", [1, 15, 16, 31, 32, 33, 100, 128, 1000, 4097])
@pytest.mark.parametrize("page", [16, 24])
def test_prefix_lengths(prefix, page):
    run(3, 5, 1, 8, 2, 64, "bf16", page, prefix, [1, 2, 17, 64, 200])


@pytest.mark.parametrize("page", [1, 2, 5, 16, 20, 32, 48, 100, 4096])
@pytest.mark.parametrize("layout", ["pages", "tokens"])
def test_page_sizes_and_layouts(page, layout):
    run(4, 3, 1, 4, 2, 64, "f16", page, 77, [1, 90, 31], layout=layout)


@pytest.mark.parametrize("n_qt", [1, 2, 3, 4, 7, 16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_draft_tokens(n_qt, dim):
    run(5, 4, n_qt, 10, 2, dim, "bf16", 16, 50, [n_qt, n_qt + 1, 40, 129])


@pytest.mark.parametrize("n_seqs", [1, 2, 7, 16, 17, 33, 64])
def test_batches(n_seqs):
    run(6, n_seqs, 1, 8, 2, 128, "bf16", 16, 300, [1 + 37 * i % 150 for i in range(n_seqs)])


def test_bound_beyond_the_lengths():
    """max_len only splits the work: a bound far above the lengths changes rounding at most."""
    q, k, v, table, lens, a = run(7, 2, 1, 4, 1, 128, "bf16", 16, 64, [30, 70])
    import torch
    wide = torch.zeros(2, 5000, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    b = B.q2_0_attn_shared(q, k, v, wide, lens, 128 ** -0.5, prefix_len=64)
    ref, tol = reference(q, k, v, table, lens, 128 ** -0.5, 1, U["bf16"])
    check(b, ref, tol)


def test_rows_that_see_nothing_are_zero():
    """A sequence of length zero, and draft queries before the first key: zeros, and the others as
    they are without them."""
    import torch
    for prefix in (0, 40):
        q, k, v, table, lens = make(8, 4, 3, 6, 2, 64, "f16", 16, prefix, [0, 1, 2, 50])
        lens = lens.clone()
        lens[0] = 0
        got = B.q2_0_attn_shared(q, k, v, table, lens, 0.125, prefix_len=prefix, n_qt=3)
        ref, tol = reference(q, k, v, table, lens, 0.125, 3, U["f16"])
        check(got, ref, tol)
        assert (got[:3] == 0).all()
        if prefix == 0:
            assert (got[3:5] == 0).all() and (got[6] == 0).all() and got[5].abs().sum() > 0


def test_lengths_inside_the_prefix():
    """Sequences shorter than the shared prefix see only their own part of it."""
    import torch
    q, k, v, table, _ = make(9, 5, 2, 8, 2, 64, "bf16", 16, 200, [10] * 5)
    lens = torch.tensor([1, 2, 33, 199, 210], dtype=torch.int32, device="cuda")
    got = B.q2_0_attn_shared(q, k, v, table, lens, 0.125, prefix_len=200, n_qt=2)
    ref, tol = reference(q, k, v, table, lens, 0.125, 2, U["bf16"])
    check(got, ref, tol)


@pytest.mark.parametrize("hole", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("page", [16, 24])
def test_unseen_places_do_not_count(hole, page):
    """NaN or inf in keys and values that some queries must not see (later draft tokens, the
    prefix past a short sequence): every query that does not see them is as if they were not there."""
    import torch
    q, k, v, table, lens = make(10, 3, 3, 6, 2, 128, "bf16", page, 40, [3, 9, 30], hole=hole)
    tab = table.cpu().numpy()
    for s, n in enumerate(lens.tolist()):                # the last token of each sequence
        for t in (k, v):
            t[int(tab[s][(n - 1) // page]), :, (n - 1) % page] = hole
    got = B.q2_0_attn_shared(q, k, v, table, lens, 128 ** -0.5, prefix_len=40, n_qt=3)
    rows = got.view(3, 3, -1)
    later = q.view(3, 3, -1).roll(1, dims=1).reshape(q.shape)       # query j as query j + 1 of the shorter sequence
    ref, tol = reference(later, k, v, table, lens - 1, 128 ** -0.5, 3, U["bf16"])
    ref, tol = (x.reshape(3, 3, -1) for x in (ref, tol))
    check(rows[:, :2], ref[:, 1:], tol[:, 1:])
    if hole != hole:
        assert torch.isnan(rows[:, 2]).all()

    q, k, v, table, _ = make(11, 2, 1, 6, 2, 128, "bf16", page, 100, [5, 5], hole=hole)
    tab = table.cpu().numpy()
    for i in range(60, 100):
        for t in (k, v):
            t[int(tab[0][i // page]), :, i % page] = hole
    lens = torch.tensor([60, 17], dtype=torch.int32, device="cuda")
    got = B.q2_0_attn_shared(q, k, v, table, lens, 128 ** -0.5, prefix_len=100)
    ref, tol = reference(q, k, v, table, lens, 128 ** -0.5, 1, U["bf16"])
    check(got, ref, tol)


def test_large_and_equal_scores():
    """Scores of some hundred units (one key takes all), equal scores, and keys all alike."""
    import torch
    run(12, 2, 1, 4, 2, 128, "bf16", 16, 40, [70, 33], spread=40.0)
    q, k, v, table, lens = make(13, 1, 1, 4, 2, 64, "f16", 16, 0, [500])
    q.zero_()
    got = B.q2_0_attn_shared(q, k, v, table, lens, 0.125)
    ref, tol = reference(q, k, v, table, lens, 0.125, 1, U["f16"])
    check(got, ref, tol)


def test_rising_scores():
    """Keys in rising order of score, so that the running reference is raised again and again."""
    import torch
    dim, n = 64, 2000
    q, k, v, table, lens = make(14, 1, 1, 2, 1, dim, "bf16", 16, 0, [n])
    q.fill_(1.0)
    tab = table.cpu().numpy()[0]
    ramp = torch.linspace(-3, 3, n, device="cuda")
    i = np.arange(n)
    k[tab[i // 16].tolist(), 0, (i % 16).tolist()] = (ramp[:, None] + 0 * k[0, 0, :1]).to(k.dtype).expand(n, dim)
    got = B.q2_0_attn_shared(q, k, v, table, lens, 1.0)
    ref, tol = reference(q, k, v, table, lens, 1.0, 1, U["bf16"])
    check(got, ref, tol)


def test_bad_lengths_and_pages_give_nan():
    import torch
    q, k, v, table, lens = make(15, 4, 1, 4, 2, 64, "bf16", 16, 32, [20, 20, 20, 20])
    lens = torch.tensor([52, -1, 1000, 52], dtype=torch.int32, device="cuda")
    table = table.clone()
    table[3, 3] = table.shape[0] * 1000                     # key 48 .. of sequence 3
    got = B.q2_0_attn_shared(q, k, v, table, lens, 0.125, prefix_len=32)
    assert torch.isnan(got[1:]).all() and torch.isfinite(got[0].float()).all()
    lens = torch.tensor([52, 40, 50, 48], dtype=torch.int32, device="cuda")    # now nobody sees it
    got = B.q2_0_attn_shared(q, k, v, table, lens, 0.125, prefix_len=32)
    assert torch.isfinite(got.float()).all()
    for page in (24,):
        q, k, v, table, lens = make(16, 2, 1, 4, 2, 64, "bf16", page, 0, [50, 60])
        table = table.clone()
        table[1, 1] = -5
        got = B.q2_0_attn_shared(q, k, v, table, lens, 0.125)
        assert torch.isnan(got[1]).all() and torch.isfinite(got[0].float()).all()


def test_empty_cache_bound():
    import torch
    q = torch.ones(2, 128, dtype=torch.float16, device="cuda")
    k = torch.zeros(1, 1, 16, 64, dtype=torch.float16, device="cuda")
    t = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    got = B.q2_0_attn_shared(q, k, k.clone(), t, torch.zeros(2, dtype=torch.int32, device="cuda"), 1.0, max_len=0)
    assert (got == 0).all()


def shared_run(seed, n_seqs, n_qt, n_q, n_kv, dim, ct, page, prefix, own, lens=None, bad=None, **kw):
    """As run, with a table wide enough (by a bound far above the lengths) that the prefix's rows of
    all sequences are taken together.  bad: (sequence row of the table, column) whose page does not exist."""
    import torch
    q, k, v, table, ln = make(seed, n_seqs, n_qt, n_q, n_kv, dim, ct, page, prefix, own, **kw)
    wide = torch.zeros(n_seqs, max(table.shape[1], 3000 // page + 1), dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    if lens is not None:
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if bad is not None:
        wide[bad[0], bad[1]] = 1 << 30
    scale = dim ** -0.5
    got = B.q2_0_attn_shared(q, k, v, wide, ln, scale, prefix_len=prefix, n_qt=n_qt)
    assert torch.equal(got.isnan(), B.q2_0_attn_shared(q, k, v, wide, ln, scale, prefix_len=prefix, n_qt=n_qt).isnan())
    ref, tol = reference(q, k, v, table, ln, scale, n_qt, U[ct])
    return got, ref, tol


@pytest.mark.parametrize("prefix", [1, 16, 31, 32, 33, 63, 64, 65, 97, 129, 300])
@pytest.mark.parametrize("page", [16, 24, 32, 48, 64])
def test_prefix_of_all_sequences(prefix, page):
    check(*shared_run(20, 5, 1, 8, 1, 128, "bf16", page, prefix, [1, 2, 17, 64, 40]))


@pytest.mark.parametrize("ct", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n_seqs,n_qt,n_q,n_kv", [(2, 1, 4, 4), (3, 1, 16, 2), (4, 4, 4, 1), (5, 1, 13, 1), (16, 1, 8, 2), (9, 2, 8, 1),
                                                  (33, 1, 8, 1)])
def test_prefix_rows(ct, dim, n_seqs, n_qt, n_q, n_kv):
    """Rows of a key head from 2 to 264: one or several waves, one or two tiles of 16 each, several workgroups."""
    own = [n_qt + 7 * i % 60 for i in range(n_seqs)]
    check(*shared_run(21, n_seqs, n_qt, n_q, n_kv, dim, ct, 16, 150, own))


@pytest.mark.parametrize("prefix", [1501, 4097, 9000])
@pytest.mark.parametrize("page", [16, 40, 256])
def test_long_prefix(prefix, page):
    check(*shared_run(22, 12, 1, 8, 1, 64, "f16", page, prefix, [1 + 31 * i % 300 for i in range(12)], layout="tokens"))


@pytest.mark.parametrize("dim,n_q", [(64, 8), (128, 4), (128, 20), (256, 4)])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("hole", [float("nan"), float("inf")])
def test_prefix_seen_in_part(dim, n_q, page, hole):
    """Sequences that end inside the prefix, one of them empty: what they do not see, NaN there too, does not
    count, and the others see it all."""
    lens = [300, 1, 0, 33, 64, 95, 310, 160]
    got, ref, tol = shared_run(23, 8, 1, n_q, 1, dim, "bf16", page, 300, [10] * 8, lens=lens)
    check(got, ref, tol)
    # the prefix from key 160 on is a hole, which sequences 0 and 6 alone see
    import torch
    q, k, v, table, _ = make(23, 8, 1, n_q, 1, dim, "bf16", page, 300, [10] * 8)
    wide = torch.zeros(8, 3000 // page + 1, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    tab = table.cpu().numpy()
    for i in range(160, 300):
        k[int(tab[0][i // page]), :, i % page] = hole
        v[int(tab[0][i // page]), :, i % page] = hole
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    holed = B.q2_0_attn_shared(q, k, v, wide, ln, dim ** -0.5, prefix_len=300)
    rows = [1, 2, 3, 4, 5, 7]
    check(holed[rows], ref[rows], tol[rows])
    if hole != hole:
        assert holed[[0, 6]].isnan().all()


@pytest.mark.parametrize("page", [16, 24, 32, 64])
@pytest.mark.parametrize("col", [0, 1, 3, 4])
def test_bad_page_in_the_prefix(page, col):
    """A prefix page that does not exist: NaN where a query sees one of its tokens, the others as ever."""
    first = col * page
    lens = [300 + 5 * i for i in range(6)] + [first, first + 1]
    got, ref, tol = shared_run(24, 8, 1, 8, 1, 128, "bf16", page, 300, [5 * i + 1 for i in range(8)], lens=lens, bad=(0, col))
    sees = [n > first for n in lens]
    assert got[sees].isnan().all()
    rest = [not s for s in sees]
    check(got[rest], ref[rest], tol[rest])


@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("prefix", [0, 100, 2000])
def test_pages_past_32_bits(page, prefix):
    """Pages whose elements lie past 2^31 in the pool: written by the append, read by the attention."""
    import torch
    n_kv, dim, seqs = 8, 128, 4
    lens = [prefix + n for n in (1, 17, 40, 90)]
    cols = -(-max(lens) // page)
    shared = prefix // page
    need = shared + seqs * (cols - shared)
    n_pages = 2 ** 32 // (n_kv * page * dim) + need + 1              # 8 GiB a pool; the last pages are used
    k, v = (torch.empty(n_pages, n_kv, page, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    own = n_pages - 1 - torch.arange(need, device="cuda")
    table = torch.cat([own[:shared].expand(seqs, -1), own[shared:].view(seqs, -1)], 1).to(torch.int32).contiguous()
    g = torch.Generator(device="cuda").manual_seed(30)
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(lens)]).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    first = torch.randn(max(lens), 2, n_kv * dim, generator=g, device="cuda")[pos.long()]        # alike at equal positions
    B.q2_0_kv_append(k, v, table, seq, pos, first[:, 0].contiguous(), first[:, 1].contiguous())
    q = torch.randn(seqs, 2 * n_kv * dim, generator=g, device="cuda").bfloat16()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = B.q2_0_attn_shared(q, k, v, table, ln, dim ** -0.5, prefix_len=prefix)
    small = (table - (n_pages - need)).contiguous()
    ks, vs = k[n_pages - need:].clone(), v[n_pages - need:].clone()
    kept = torch.zeros(need, page, dtype=torch.bool, device="cuda")
    kept[small[seq.long(), (pos // page).long()].long(), (pos % page).long()] = True
    for t in (ks, vs):
        t.transpose(1, 2)[~kept] = 0
    ref, tol = reference(q, ks, vs, small, ln, dim ** -0.5, 1, U["bf16"])
    check(got, ref, tol)


def test_row_strides_and_streams():
    """Strided q rows, and a call on another stream than the tensors' own."""
    import torch
    q, k, v, table, lens = make(17, 3, 1, 4, 2, 64, "bf16", 16, 20, [30, 40, 9])
    wide = torch.zeros(3, 4 * 64 + 40, dtype=q.dtype, device="cuda")
    wide[:, 16 : 16 + 256] = q
    ref, tol = reference(q, k, v, table, lens, 0.125, 1, U["bf16"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = B.q2_0_attn_shared(wide[:, 16 : 16 + 256], k, v, table, lens, 0.125, prefix_len=20)
    st.synchronize()
    check(got, ref, tol)


def test_refusals():
    import torch
    q, k, v, table, lens = make(18, 2, 1, 4, 2, 64, "bf16", 16, 20, [30, 40])
    with pytest.raises(ValueError):
        B.q2_0_attn_shared(q.half(), k, v, table, lens, 0.125)
    with pytest.raises(ValueError):
        B.q2_0_attn_shared(q[:, :100], k, v, table, lens, 0.125)
    with pytest.raises(ValueError):
        B.q2_0_attn_shared(q, k, v, table, lens[:1], 0.125)
    with pytest.raises(ValueError):
        B.q2_0_attn_shared(q, k, v, table.long(), lens, 0.125)
    with pytest.raises(ValueError):
        B.q2_0_attn_shared(q[:1], k, v, table, lens, 0.125)
    for kw in (dict(scale=0.0), dict(scale=0.1, prefix_len=500), dict(scale=0.1, max_len=10 ** 6)):
        with pytest.raises(B.Q2_0Error):
            B.q2_0_attn_shared(q, k, v, table, lens, **kw)
