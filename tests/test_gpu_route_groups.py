"""Expert choice from biased scores inside the best groups, against the definition in 64 bits: ids exactly, weights to their
one rounding to float32."""

import numpy as np
import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

SCORE = {"softmax": B.Q2_0_SCORE_SOFTMAX, "sigmoid": B.Q2_0_SCORE_SIGMOID}


def types():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def largest_first(x):
    """Places of a row's values, largest first, the lower place first among equals, NaN last."""
    return np.lexsort((np.arange(x.shape[1])[None].repeat(x.shape[0], 0), -np.where(np.isnan(x), -np.inf, x), np.isnan(x)), axis=1)


def reference(x, used, score, bias, n_group, n_used, top, normalise, scale):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-x))
        else:
            most = np.fmax.reduce(x, axis=1, keepdims=True)
            e = np.exp(x - np.where(most == -np.inf, 0, most))
            total = e.sum(1, keepdims=True)
            s = np.where(total == 0, 0, e / total)
        b = s if bias is None else s + bias
        t, n = b.shape
        g = b.reshape(t * n_group, n // n_group)
        best = np.take_along_axis(g, largest_first(g), 1)[:, :top].sum(1).reshape(t, n_group)
        open_ = np.zeros((t, n_group), bool)
        np.put_along_axis(open_, largest_first(best)[:, :n_used], True, 1)
        # closed experts come after everything, NaN included
        shut = ~open_.repeat(n // n_group, 1)
        order = np.lexsort((np.arange(n)[None].repeat(t, 0), -np.where(np.isnan(b), -np.inf, b), np.isnan(b), shut), axis=1)
        ids = order[:, :used]
        w = np.take_along_axis(s, ids, 1)
        if bias is not None:
            w = np.where(bias[ids] == -np.inf, 0, w)
        if normalise:
            total = w.sum(1, keepdims=True)
            w = np.where(total == 0, 0, w / total)
        return ids, w * scale


def check(logits, used, score="sigmoid", bias=None, n_group=1, n_used=1, top=1, normalise=True, scale=1.0):
    import torch
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids, w = B.q2_0_moe_route_groups(logits, used, SCORE[score], bias=b, n_group=n_group, n_group_used=n_used, group_top=top,
                                     normalise=normalise, scale=scale)
    torch.cuda.synchronize()
    rid, rw = reference(logits.double().cpu().numpy(), used, score, None if bias is None else np.float64(np.float32(bias)), n_group,
                        n_used, top, normalise, np.float64(np.float32(scale)))
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    # one rounding to float32 (2^-24, below the normal range 2^-150); the 64-bit steps before it are some 2^-50
    ok = ~np.isnan(rw)
    assert np.all(np.abs(got - rw)[ok] <= (2.0 ** -24 + 2.0 ** -45) * np.abs(rw)[ok] + 2.0 ** -150)
    return ids.cpu().numpy(), got


def logits_of(t, n, x="f32", seed=0, spread=1.5, pad=0, off=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = (spread * torch.randn(t * (n + pad) + off, generator=g, device="cuda")).to(types()[x])
    return buf[off:].view(t, n + pad)[:, :n]


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,picked,top", [(8, 1, 1, 1), (60, 5, 3, 1), (64, 8, 4, 2), (128, 8, 4, 2), (256, 8, 4, 2),
                                                 (250, 5, 2, 2), (320, 64, 7, 1), (1024, 32, 9, 2), (1000, 1, 1, 2)])
def test_sizes(x, score, n, groups, picked, top):
    bias = 0.1 * np.random.default_rng(n).standard_normal(n)
    for normalise, b in ((True, bias), (False, None)):
        check(logits_of(37, n, x, seed=n), min(8, picked * (n // groups)), score, b, groups, picked, top, normalise, 2.5)


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 4099])
def test_token_counts(tokens):
    check(logits_of(tokens, 160, seed=tokens), 6, "sigmoid", np.linspace(-0.2, 0.2, 160), 8, 3, 2)


@pytest.mark.parametrize("used", [1, 2, 63, 64])
def test_choices(used):
    check(logits_of(9, 64, seed=used), used, "softmax", None, 4, 4, 2)
    check(logits_of(9, 512, seed=used), used, "sigmoid", None, 8, 1 if used <= 64 else 2, 1)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("pad,off", [(1, 0), (0, 1), (7, 3)])
def test_rows_of_any_alignment(x, pad, off):
    check(logits_of(11, 96, x, seed=pad, pad=pad, off=off), 5, "sigmoid", np.zeros(96), 6, 2, 2)


def test_equal_scores_go_by_index():
    import torch
    x = torch.zeros(3, 256, device="cuda")
    ids, _ = check(x, 8, "softmax", None, 8, 4, 2)
    assert np.array_equal(ids, np.arange(8)[None].repeat(3, 0))
    x[1, 200] = x[1, 40] = 1.0
    ids, _ = check(x, 8, "sigmoid", None, 8, 2, 1)
    assert ids[1].tolist() == [40, 200, 32, 33, 34, 35, 36, 37]
    check(logits_of(200, 128, "bf16", spread=0.02), 8, "sigmoid", None, 4, 2, 2)      # many equal values
    check(logits_of(200, 128, spread=60.0), 8, "sigmoid", None, 4, 2, 2)              # sigmoids of 0 and of 1
    check(logits_of(200, 128, spread=600.0), 8, "softmax", None, 4, 2, 2)             # all but a few underflow


def test_scores_that_32_bits_do_not_tell_apart():
    """Logits one float32 step apart about 9: their sigmoids are the same float32, and a bias of the size of a step decides
    elsewhere."""
    import torch
    x = torch.full((1, 64), -3.0, device="cuda")
    step = 2.0 ** -20
    for i in range(8):
        x[0, 10 + i] = 9.0 + step * i
    ids, _ = check(x, 8, "sigmoid")
    assert ids[0].tolist() == [17, 16, 15, 14, 13, 12, 11, 10]
    bias = np.zeros(64)
    bias[12] = 2.0 ** -30                      # more than the distance of two sigmoids (1e-4 * 2^-20) times 8
    ids, _ = check(x, 3, "sigmoid", bias)
    assert ids[0].tolist() == [12, 17, 16]


def test_masks():
    import torch
    inf = float("inf")
    x = logits_of(6, 32)
    bias = np.zeros(32)
    bias[4:] = -inf                            # four experts are left, six are chosen
    ids, w = check(x, 6, "sigmoid", bias, 4, 2, 2)
    assert np.all(np.sort(ids[:, :4]) == np.arange(4)) and np.all(w[:, 4:] == 0) and np.allclose(w.sum(1), 1)
    ids, w = check(x, 3, "softmax", np.full(32, -inf), 4, 2, 2)
    assert np.all(ids == np.arange(3)) and np.all(w == 0)
    x = torch.full((2, 32), -inf, device="cuda")
    x[1, 9] = 0.0
    for score in ("softmax", "sigmoid"):
        for b in (None, np.linspace(0, 1, 32)):
            ids, w = check(x, 4, score, b, 4, 2, 1)
            assert np.all(w[0] == 0)
    x = logits_of(8, 32, seed=3)
    x[0, 3] = x[1, 0] = x[5, 30] = float("nan")
    x[2, 7] = inf
    x[3] = float("nan")
    x[4, :] = inf
    x[6, ::2] = -inf
    for score in ("softmax", "sigmoid"):
        for normalise in (True, False):
            check(x, 5, score, None, 4, 2, 2, normalise)
            check(x, 5, score, np.linspace(-1, 1, 32), 4, 3, 1, normalise)
            check(x, 32, score, None, 4, 4, 1, normalise)


def test_results_given_and_rows_after_them():
    import torch
    x = logits_of(5, 64)
    ids, w = torch.full((7, 4), -9, dtype=torch.int32, device="cuda"), torch.full((7, 4), -9.0, device="cuda")
    got = B.q2_0_moe_route_groups(x, 4, ids=ids[:5], weights=w[:5])
    torch.cuda.synchronize()
    assert got[0].data_ptr() == ids.data_ptr() and torch.all(ids[5:] == -9) and torch.all(w[5:] == -9)
    rid, _ = reference(x.double().cpu().numpy(), 4, "sigmoid", None, 1, 1, 1, True, 1.0)
    assert np.array_equal(ids[:5].cpu().numpy(), rid)


def test_the_chosen_feed_the_expert_layer():
    """ids and weights go straight into the expert layer: without a bias, groups or sigmoid they are q2_0_moe_route's."""
    import torch
    x = logits_of(6, 16)
    a = B.q2_0_moe_route(x, 4)
    b = B.q2_0_moe_route_groups(x, 4, B.Q2_0_SCORE_SOFTMAX)
    assert torch.equal(a[0], b[0])
    # exp, sum and quotient in float32 there: a few roundings
    assert torch.all((a[1] - b[1]).abs() <= 8 * 2.0 ** -24 * b[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_expert(score):
    import torch
    x = torch.tensor([[0.3], [-2.0], [40.0]], device="cuda")
    ids, w = B.q2_0_moe_route_groups(x, 1, SCORE[score], bias=torch.tensor([0.25], device="cuda"), normalise=False)
    want = 1 / (1 + np.exp(-x.double().cpu().numpy())) if score == "sigmoid" else np.ones((3, 1))
    assert ids.tolist() == [[0]] * 3
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= (2.0 ** -24 + 2.0 ** -45) * want)
