"""Attention where one key leads by many powers of two and the tens of thousands behind it, each of a
weight that a 16-bit type barely holds, make up the result: the leading key's value is zero."""

import math

import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

# A weight errs by half a unit of its type, or by half of the type's least step, of the greatest weight at most:
# f16's 2^-24 with the factor 2^11 that weights carry; the sum below the line takes the same weights.
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
STEP = {"f16": 2.0 ** -36, "bf16": 2.0 ** -130}


@pytest.mark.parametrize("ct", ["f16", "bf16"])
@pytest.mark.parametrize("lead_at", ["first", "last"])
@pytest.mark.parametrize("n_seqs,prefix", [(1, 0), (5, 40000)])
@pytest.mark.parametrize("lead", [12.0, 25.5, 30.0])
def test_many_keys_behind_a_leading_one(ct, lead_at, n_seqs, prefix, lead):
    import torch
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[ct]
    dim, page, keys = 64, 64, 40000
    n = keys + (1 if prefix else 0)                          # (a key of its own for each sequence)
    g = torch.Generator(device="cuda").manual_seed(40)
    pages = -(-n // page)
    # queries of ones, and of the leading key one element: its score is lead powers of two above the others', which are 0
    q = torch.ones(n_seqs, dim, device="cuda").to(dt)
    k = torch.zeros(pages, 1, page, dim, device="cuda").to(dt)
    v = (0.5 + torch.rand(k.shape, generator=g, device="cuda")).to(dt)
    at = 0 if lead_at == "first" else keys - 1
    k[at // page, 0, at % page, 0] = 1.0
    v[at // page, 0, at % page] = 0.0
    scale = lead * math.log(2.0)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(n_seqs, -1).contiguous()
    lens = torch.full((n_seqs,), n, dtype=torch.int32, device="cuda")
    got = B.q2_0_attn_shared(q, k, v, table, lens, scale, prefix_len=prefix, max_len=n).double()
    vs = v.double().view(-1, dim)[:n]
    p = torch.full((n, 1), 2.0 ** -lead, dtype=torch.float64, device="cuda")
    p[at] = 1.0
    p /= p.sum()
    ref = (p * vs).sum(0)
    # scores: products of one term, the scale and the exponent's f32 product and sum round, on lead + 11 units at most
    delta = 4 * 2.0 ** -24 * (lead + 11) + n * 2.0 ** -24
    tol = (2 * U[ct] + 2 * delta) * ref + n * STEP[ct] * (1.5 + ref) + 2.0 ** -25
    err = (got - ref).abs()
    assert torch.isfinite(err).all() and (err <= tol).all(), "worst %.3g of its tolerance" % (err / tol).max().item()
    assert (ref > 10 * tol).all()                            # the keys behind are what the result consists of
