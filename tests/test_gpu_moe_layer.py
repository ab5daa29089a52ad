"""Expert choice and the whole expert layer against their definitions in 64 bits."""

import numpy as np
import pytest

import oracle
from ternary_bit_quantized_amd import q2_0 as B
from ternary_bit_quantized_amd import synth

pytestmark = pytest.mark.gpu


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------------------- choice

def choice(x, used, normalise):
    x = x.astype(np.float64)
    key = np.where(np.isnan(x), -np.inf, x)
    # NaN after -inf: two sorts, the last by value
    ids = np.lexsort((np.arange(x.shape[1])[None].repeat(x.shape[0], 0), np.isnan(x), -key), axis=1)[:, :used]
    v = np.take_along_axis(x, ids, 1)
    m = v[:, :1]
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp(v - m)
        s = e.sum(1, keepdims=True) if normalise else np.exp(x - m).sum(1, keepdims=True)
        w = e / s
    w[m[:, 0] == -np.inf] = 0.0
    return ids, w, np.abs(v - m)


def check_choice(x, used, normalise, xt=None):
    import torch
    t = dev(x) if xt is None else dev(x).to(xt)
    ids, w = B.q2_0_moe_route(t, used, normalise=normalise)
    rid, rw, dist = choice(t.double().cpu().numpy() if xt is not None else x, used, normalise)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    # exp of a rounded difference (|l - m| 2^-24), the exponential itself and the quotient (4 units), a sum
    # over up to 8 terms a lane and 6 joins, its terms' errors included
    far = np.where(np.isfinite(dist), dist, 0)
    tol = rw * 2.0 ** -24 * (2 * far + 24 + x.shape[1] / 64) + 2.0 ** -126
    ok = ~np.isnan(rw)
    assert np.all(np.abs(got - rw)[ok] <= tol[ok]), np.max((np.abs(got - rw) / tol)[ok])


@pytest.mark.parametrize("n", [1, 2, 8, 60, 64, 65, 128, 129, 160, 256, 257, 384, 1024, 1025, 8192])
@pytest.mark.parametrize("normalise", [True, False])
def test_choice_sizes(n, normalise):
    rng = np.random.default_rng(n)
    for used in sorted({1, min(n, 3), min(n, 8), min(n, 64)}):
        check_choice(rng.standard_normal((5, n)).astype(np.float32) * 2, used, normalise)


@pytest.mark.parametrize("tokens", [1, 3, 4, 5, 1001])
def test_choice_tokens(tokens):
    check_choice(np.random.default_rng(tokens).standard_normal((tokens, 128)).astype(np.float32), 8, True)


def test_choice_types():
    import torch
    x = np.random.default_rng(1).standard_normal((33, 128)).astype(np.float32)
    for xt in (torch.float16, torch.bfloat16):       # many equal values: the lower index first
        check_choice(x, 8, True, xt)


def test_choice_ties_and_special_values():
    x = np.zeros((9, 70), np.float32)
    x[1, :] = -np.inf                               # nothing left: weights 0
    x[2, ::2] = -np.inf                             # half masked
    x[3, 5:] = np.finfo(np.float32).min             # masked by the type's lowest value
    x[4, 3] = np.nan
    x[5, :] = np.nan
    x[6, :] = -np.inf
    x[6, 69] = 1.0
    x[7, ::3] = -0.0                                # -0 and +0 are equal
    x[8] = np.repeat(np.arange(7), 10)
    for normalise in (True, False):
        check_choice(x, 8, normalise)


def test_choice_strided_and_refusals():
    import torch
    x = np.random.default_rng(2).standard_normal((6, 200)).astype(np.float32)
    t = dev(x)[:, 3:131]
    ids, _ = B.q2_0_moe_route(t, 4)
    assert np.array_equal(ids.cpu().numpy(), choice(x[:, 3:131], 4, True)[0])
    for bad in (lambda: B.q2_0_moe_route(dev(x).double(), 4), lambda: B.q2_0_moe_route(dev(x).t(), 4),
                lambda: B.q2_0_moe_route(dev(x), 4, weights=torch.zeros(6, 5, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for used in (0, 65, 201):
        with pytest.raises(B.Q2_0Error):
            B.q2_0_moe_route(dev(x), used)


# -------------------------------------------------------------------------------- layer

def experts(seed, ne, M, K):
    return np.stack([synth.weight(seed, e, 0, M, K, "tern_c3", synth.ScaleDist("loguniform", 1e-3, 1e-1, 0.01))
                     for e in range(ne)])


REL = 1e-5      # each product's contract: 1e-5 * sum |W x|


def layer(wg, wu, wd, ff, K, x, ids, weights):
    """(y, tolerance): the definition on the oracle's fp64 products, and the products' bounds carried through."""
    y, tol = np.zeros((len(x), K)), np.zeros((len(x), K))
    for t in range(len(x)):
        for u, e in enumerate(ids[t]):
            if e < 0 or e >= len(wg):
                y[t] = np.nan
                continue
            g, ag = (a[0] for a in oracle.mul_mat(wg[e], ff, K, x[t:t + 1]))
            p, ap = (a[0] for a in oracle.mul_mat(wu[e], ff, K, x[t:t + 1]))
            s = g / (1 + np.exp(-g))
            h = s * p
            # |silu'| < 1.1; silu and the product in f32: 6 roundings and an exponential off by its argument's
            dh = 1.1 * REL * ag * np.abs(p) + REL * ap * np.abs(s) + 2.0 ** -23 * (4 + np.abs(g)) * np.abs(h)
            h32 = h.astype(np.float32)
            z, az = (a[0] for a in oracle.mul_mat(wd[e], K, ff, h32[None]))
            dz = oracle.mul_mat(wd[e], K, ff, (dh + 2.0 ** -24 * np.abs(h)).astype(np.float32)[None])[1][0]
            w = float(weights[t, u])
            y[t] += w * z
            tol[t] += abs(w) * (REL * az + dz) + 2.0 ** -23 * len(ids[t]) * abs(w) * np.abs(z)
    return y, tol * (1 + 1e-3) + 1e-30


def run(seed, tokens, ne, used, ff, K, xt="f32", ids=None, shift=0, ldx=0, weights=None):
    import torch
    rng = np.random.default_rng(seed)
    wg, wu, wd = (experts(seed + i, ne, *s) for i, s in enumerate(((ff, K), (ff, K), (K, ff))))
    x = synth.activations(seed, 0, 0, tokens, K)
    if ids is None:
        ids = np.stack([rng.permutation(ne)[:used] for _ in range(tokens)]) if used <= ne else rng.integers(0, ne, (tokens, used))
    ids = np.asarray(ids, np.int32)
    if weights is None:
        weights = rng.dirichlet(np.ones(max(1, ids.shape[1])), tokens).astype(np.float32)[:, : ids.shape[1]]
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[xt]
    xd = torch.zeros(tokens, K + ldx, dtype=dt, device="cuda")[:, :K]
    xd.copy_(dev(x))
    x = xd.float().cpu().numpy()

    def put(w):                                    # at a 2-byte offset where asked
        b = torch.zeros(w.size + 16, dtype=torch.uint8, device="cuda")
        b[shift : shift + w.size] = dev(w.reshape(-1))
        return b[shift : shift + w.size]

    yd = torch.full((tokens, K + 5), float("inf"), device="cuda")
    need = B.moe_layer_workspace_bytes(ff, K, ids.shape[1], tokens)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    args = (put(wg), put(wu), put(wd), ne, ff, K, xd, dev(ids), dev(weights))
    got = B.q2_0_moe_layer(*args, y=yd[:, :K], workspace=ws)
    torch.cuda.synchronize()
    assert torch.isinf(yd[:, K:]).all(), "wrote past a row"
    y, tol = layer(wg, wu, wd, ff, K, x, ids, weights)
    g = got.double().cpu().numpy()
    bad = np.isnan(y)
    assert np.array_equal(np.isnan(g), bad)
    err = np.abs(g - y)
    assert np.all(err[~bad] <= tol[~bad]), "worst %.3g of its tolerance" % np.max((err / tol)[~bad])
    assert torch.equal(torch.nan_to_num(B.q2_0_moe_layer(*args)), torch.nan_to_num(got)), "two runs differ"


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 8, 9, 16, 33, 64])
def test_layer_tokens(tokens):
    run(tokens, tokens, 10, 3, 128, 192)


@pytest.mark.parametrize("ff,K", [(64, 64), (64, 1088), (704, 1600), (768, 2048), (1088, 64), (192, 4160), (1024, 1024)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_layer_sizes(ff, K, xt):
    run(ff + K, 3, 4, 2, ff, K, xt=xt)


@pytest.mark.parametrize("xt", ["f32", "f16", "bf16"])
def test_layer_types_and_unaligned(xt):
    for shift, ldx in ((0, 4), (2, 1), (6, 3), (8, 0)):
        run(7, 5, 6, 2, 192, 320, xt=xt, shift=shift, ldx=ldx)


@pytest.mark.parametrize("used", [1, 2, 8, 32])
def test_layer_used(used):
    run(used, 4, 40, used, 64, 128)


def test_layer_one_expert_takes_all():
    run(3, 20, 4, 2, 128, 128, ids=np.full((20, 2), 1))                 # more pairs than a pass takes, ids that repeat
    run(4, 64, 2, 1, 64, 64, ids=np.zeros((64, 1)))
    run(5, 1, 8, 4, 64, 64, ids=[[7, 7, 7, 7]])


def test_layer_many_pairs():
    """The most tokens with the most experts each, some experts chosen far more often than others, a token's twice."""
    rng = np.random.default_rng(70)
    ids = np.minimum(rng.geometric(0.08, (64, 32)) - 1, 39)
    run(70, 64, 40, 32, 64, 64, ids=ids)
    ids[rng.random(ids.shape) < 0.3] = -1                              # most tokens are NaN then; the others not
    ids[10:20] = np.arange(32)
    run(71, 64, 40, 32, 64, 128, ids=ids)


@pytest.mark.parametrize("ne", [300, 8192])
def test_layer_many_experts(ne):
    """More experts than pairs, few of them chosen, the last among them."""
    ff, K, tokens = 64, 64, 33
    few = [experts(80 + i, 8, *s) for i, s in enumerate(((ff, K), (ff, K), (K, ff)))]
    wg, wu, wd = (np.concatenate([w] * (ne // 8 + 1))[:ne] for w in few)
    rng = np.random.default_rng(ne)
    ids = rng.integers(0, ne, (tokens, 2)).astype(np.int32)
    ids[::5, 0], ids[1::7, 1] = ne - 1, 0
    w = rng.dirichlet(np.ones(2), tokens).astype(np.float32)
    x = synth.activations(81, 0, 0, tokens, K)
    got = B.q2_0_moe_layer(dev(wg), dev(wu), dev(wd), ne, ff, K, dev(x), dev(ids), dev(w)).double().cpu().numpy()
    y, tol = layer(wg, wu, wd, ff, K, x, ids, w)
    assert np.all(np.abs(got - y) <= tol)


def test_layer_ids_out_of_range():
    ids = np.array([[0, 1], [-1, 2], [3, 4], [2, 0], [1000000, -5]])
    run(6, 5, 4, 2, 128, 192, ids=ids)


def test_layer_zero_weights_and_no_experts():
    import torch
    run(8, 3, 4, 2, 64, 64, weights=np.zeros((3, 2), np.float32))
    x = torch.ones(3, 64, device="cuda")
    w = torch.zeros(4 * 64 * 18, dtype=torch.uint8, device="cuda")
    y = B.q2_0_moe_layer(w, w, w, 4, 64, 64, x, torch.zeros(3, 0, dtype=torch.int32, device="cuda"),
                         torch.zeros(3, 0, device="cuda"))
    assert (y == 0).all()


def test_layer_activation_range():
    """Tokens 2^40 apart share an expert: each is scaled by itself."""
    import torch
    ff, K = 128, 256
    wg, wu, wd = (experts(20 + i, 2, *s) for i, s in enumerate(((ff, K), (ff, K), (K, ff))))
    x = synth.activations(20, 0, 0, 4, K)
    x[1] *= 2.0 ** -30
    x[2] *= 2.0 ** 10
    ids, w = np.zeros((4, 1), np.int32), np.ones((4, 1), np.float32)
    got = B.q2_0_moe_layer(dev(wg), dev(wu), dev(wd), 2, ff, K, dev(x), dev(ids), dev(w)).double().cpu().numpy()
    y, tol = layer(wg, wu, wd, ff, K, x, ids, w)
    assert np.all(np.abs(got - y) <= tol)


def test_layer_nan_token_stays_alone():
    import torch
    ff, K = 64, 128
    wg, wu, wd = (experts(30 + i, 2, *s) for i, s in enumerate(((ff, K), (ff, K), (K, ff))))
    x = synth.activations(30, 0, 0, 3, K)
    ids, w = np.zeros((3, 1), np.int32), np.ones((3, 1), np.float32)
    y, tol = layer(wg, wu, wd, ff, K, x, ids, w)
    x[1, 5] = np.nan
    got = B.q2_0_moe_layer(dev(wg), dev(wu), dev(wd), 2, ff, K, dev(x), dev(ids), dev(w)).double().cpu().numpy()
    assert np.isnan(got[1]).all()
    assert np.all(np.abs(got - y)[[0, 2]] <= tol[[0, 2]])


@pytest.mark.parametrize("tokens", [1, 33])
def test_layer_outlier_at_the_limit(tokens):
    """One activation so large that max|x| sum|W| is 0.9 of the 2^12 times sum|W x| of every row that the fixed-point
    contract allows: where its weight is 0 the other products keep their accuracy."""
    ff, K, ne = 64, 128, 3
    rng = np.random.default_rng(40)

    def mat(rows, cols):                       # the first column's weights 0, the others +-1 by the same scale
        codes = rng.choice([0, 2], size=(ne * rows, cols)).astype(np.uint8)
        codes[:, 0] = 1
        return synth.pack(codes, np.full((ne * rows, cols // 64), 0.05, np.float16)).reshape(ne, rows, -1)

    wg, wu, wd = mat(ff, K), mat(ff, K), mat(K, ff)
    x = rng.uniform(0.5, 1.0, (tokens, K)).astype(np.float32)
    # sum|W| = 127 * 0.05, sum|W x| >= 127 * 0.05 * 0.5
    x[:, 0] = 0.9 * 2.0 ** 12 * 0.5
    ids = rng.integers(0, ne, (tokens, 2)).astype(np.int32)
    w = rng.dirichlet(np.ones(2), tokens).astype(np.float32)
    got = B.q2_0_moe_layer(dev(wg), dev(wu), dev(wd), ne, ff, K, dev(x), dev(ids), dev(w)).double().cpu().numpy()
    y, tol = layer(wg, wu, wd, ff, K, x, ids, w)
    assert np.all(np.abs(got - y) <= tol), np.max(np.abs(got - y) / tol)


def test_layer_weights_past_32_bits():
    """Experts that lie more than 4 GiB into their tensors give what they give in small ones."""
    import torch
    ff, K, ne = 1024, 4096, 3700                       # 1.18 MB an expert's matrix, 4.4 GB in all
    nb = ff * K // 64 * 18
    wg, wu, wd = (experts(50 + i, 2, *s) for i, s in enumerate(((ff, K), (ff, K), (K, ff))))
    big = []
    for w in (wg, wu, wd):
        b = torch.zeros(ne * nb, dtype=torch.uint8, device="cuda")
        b[(ne - 2) * nb:] = dev(w.reshape(-1))
        big.append(b)
    assert (ne - 2) * nb > 2 ** 32
    for tokens in (1, 40):
        x = dev(synth.activations(51, 0, 0, tokens, K))
        ids = torch.zeros(tokens, 2, dtype=torch.int32, device="cuda")
        ids[:, 1] = 1
        w = torch.full((tokens, 2), 0.5, device="cuda")
        small = B.q2_0_moe_layer(dev(wg), dev(wu), dev(wd), 2, ff, K, x, ids, w)
        got = B.q2_0_moe_layer(*big, ne, ff, K, x, ids + (ne - 2), w)
        if tokens == 1:
            assert torch.equal(got, small)
        else:                                           # (the larger expert count may take fewer pairs a pass)
            size = small.abs().max()
            assert (got - small).abs().max() <= 2e-6 * size


def test_layer_and_choice_on_another_stream():
    import torch
    ff, K, ne = 128, 192, 6
    wg, wu, wd = (dev(experts(60 + i, ne, *s)) for i, s in enumerate(((ff, K), (ff, K), (K, ff))))
    x = dev(synth.activations(60, 0, 0, 33, K))
    logits = dev(synth.activations(61, 0, 0, 33, 64))[:, :ne].contiguous()
    want_ids, want_w = B.q2_0_moe_route(logits, 2)
    want = B.q2_0_moe_layer(wg, wu, wd, ne, ff, K, x, want_ids, want_w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ids, w = (torch.empty_like(t) for t in (want_ids, want_w))
    y = torch.empty_like(want)
    ws = torch.empty(B.moe_layer_workspace_bytes(ff, K, 2, 33), dtype=torch.uint8, device="cuda")
    B.q2_0_moe_route(logits, 2, ids=ids, weights=w, stream=st.cuda_stream)
    B.q2_0_moe_layer(wg, wu, wd, ne, ff, K, x, ids, w, y=y, workspace=ws, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w) and torch.equal(y, want)


def test_layer_refusals():
    import torch
    x = torch.zeros(3, 64, device="cuda")
    w = torch.zeros(4 * 64 * 18, dtype=torch.uint8, device="cuda")
    ids, ws = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, device="cuda")
    with pytest.raises(ValueError):
        B.q2_0_moe_layer(w[:100], w, w, 4, 64, 64, x, ids, ws)
    with pytest.raises(ValueError):
        B.q2_0_moe_layer(w, w, w, 4, 64, 64, x, ids.long(), ws)
    with pytest.raises(ValueError):
        B.q2_0_moe_layer(w, w, w, 4, 64, 64, x, ids, ws[:2])
    with pytest.raises(ValueError):
        B.q2_0_moe_layer(w, w, w, 4, 64, 64, x.double(), ids, ws)
    big = torch.zeros(65, 64, device="cuda")
    with pytest.raises(B.Q2_0Error):
        B.q2_0_moe_layer(w, w, w, 4, 64, 64, big, torch.zeros(65, 1, dtype=torch.int32, device="cuda"),
                         torch.zeros(65, 1, device="cuda"))
