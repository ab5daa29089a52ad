"""Attention whose result is the small difference of two nearly equal halves of the softmax weights: half of
the keys have value 1 and score 0, the others value -1 and a score a little below."""

import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

# A weight is held as its value in the cache's type and what that left: half a unit squared.  The result is rounded
# once, to a unit at most.
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
WEIGHT = {"f16": 2.0 ** -24, "bf16": 2.0 ** -18}


@pytest.mark.parametrize("ct", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("prefix,lens", [(0, [2, 64, 770]), (320, [322, 400, 1090]), (320, [2, 34, 100, 322, 1090])])
def test_difference_of_nearly_equal_halves(ct, dim, prefix, lens):
    import torch
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[ct]
    page, heads, n = 32, 12, len(lens)
    cols = 3000 // page + 1                                  # (a bound far above the lengths: the prefix is taken for all at once)
    k = torch.zeros(cols, 1, page, dim, device="cuda").to(dt)
    k[:, :, 1::2, 0] = -1.0
    v = torch.ones_like(k)
    v[:, :, 1::2] = -1.0
    q = torch.zeros(n, heads, dim, device="cuda")
    gap = torch.logspace(-3, 0, n * heads, device="cuda").view(n, heads).to(dt)
    q[:, :, 0] = gap.float()
    table = torch.arange(cols, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()
    got = B.q2_0_attn_shared(q.to(dt).view(n, -1), k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1.0,
                             prefix_len=prefix).double().view(n, heads, dim)
    p = torch.exp(-gap.double())
    ref = ((1 - p) / (1 + p))[:, :, None]
    # scores are one product; scale, exponent and the f32 sums round
    delta = 4 * 2.0 ** -24 + max(lens) * 2.0 ** -24
    tol = 2 * WEIGHT[ct] + 2 * delta + U[ct] * ref + 2.0 ** -24
    err = (got - ref).abs()
    assert torch.isfinite(err).all() and (err <= tol).all(), "worst %.3g of its tolerance" % (err / tol).max().item()
