"""An infinite value that a query sees makes its result infinite in that element, of the same sign, and leaves the
other elements and the queries that do not see it alone."""

import pytest
from test_gpu_attn_shared import U, check, make, reference

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ct", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("prefix,wide,lens", [(0, 0, [40, 90, 700]), (200, 3000, [210, 250, 231]), (200, 3000, [20, 101, 250])])
def test_infinite_values(ct, dim, prefix, wide, lens):
    import torch
    n, page, n_q, n_kv = len(lens), 16, 4, 2
    # (scores of a few units at most, so that no weight is below 2^-24 of its row's largest)
    q, k, v, table, _ = make(70, n, 1, n_q, n_kv, dim, ct, page, prefix, [max(1, m - prefix) for m in lens], spread=0.5, hole=0.0)
    table = torch.nn.functional.pad(table, (0, max(0, wide // page - table.shape[1]))).contiguous()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref, tol = reference(q, k, v, table, ln, dim ** -0.5, 1, U[ct])
    inf = float("inf")
    # sequence s sees keys of the prefix and its own; elements 0 and 5 of key head 0 at key 10, 7 of head 1 at key 100
    for key, head, at, value in ((10, 0, 0, inf), (10, 0, 5, -inf), (100, 1, 7, inf)):
        for row in table[:1] if key < prefix else table:
            v[int(row[key // page]), head, key % page, at] = value
    got = B.q2_0_attn_shared(q, k, v, table, ln, dim ** -0.5, prefix_len=prefix).double().cpu()
    got = got.view(n, n_kv, n_q // n_kv, dim)
    ref, tol = (torch.from_numpy(t).view(got.shape).clone() for t in (ref, tol))
    for s, length in enumerate(lens):
        if length > 10:
            assert (got[s, 0, :, 0] == inf).all() and (got[s, 0, :, 5] == -inf).all()
            got[s, 0, :, 0], got[s, 0, :, 5], ref[s, 0, :, 0], ref[s, 0, :, 5] = 0, 0, 0, 0
        if length > 100:
            assert (got[s, 1, :, 7] == inf).all()
            got[s, 1, :, 7], ref[s, 1, :, 7] = 0, 0
    check(got, ref.numpy(), tol.numpy())
