"""Calls on a stream that is not the current one and that make their workspace and results themselves: the
same results as on the current stream, though the current stream allocates and writes right after the call."""

import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["stream", "handle", "default stream"])
def test_own_buffers_on_another_stream(form, monkeypatch):
    import torch
    g = torch.Generator(device="cuda").manual_seed(50)
    n, heads, kv, dim, page, pre = 6, 8, 2, 64, 16, 3000
    cols = pre // page + 4
    k, v = (torch.randn(cols, kv, page, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(n, heads * dim, generator=g, device="cuda").bfloat16()
    table = torch.arange(cols, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()
    lens = torch.full((n,), pre + 40, dtype=torch.int32, device="cuda")
    ne, ff, K, tok, used = 16, 256, 512, 20, 4
    up, gate = (B.q2_0_quantize(torch.randn(ne * ff, K, generator=g, device="cuda")) for _ in range(2))
    down = B.q2_0_quantize(torch.randn(ne * K, ff, generator=g, device="cuda"))
    x = torch.randn(tok, K, generator=g, device="cuda")
    logits = torch.randn(tok, ne, generator=g, device="cuda")

    workspaces = []
    for name, at in (("attn_shared_raw", 15), ("moe_layer_raw", 15)):
        monkeypatch.setattr(B, name, lambda *a, raw=getattr(B, name), at=at: workspaces.append(a[at:at + 2]) or raw(*a))

    def calls(stream):
        ids, weights = B.q2_0_moe_route(logits, used, stream=stream)
        att = B.q2_0_attn_shared(q, k, v, table, lens, 0.125, prefix_len=pre, stream=stream)
        y = B.q2_0_moe_layer(gate, up, down, ne, ff, K, x, ids, weights, stream=stream)
        return ids, weights, att, y

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream, current = {"stream": (side, None), "handle": (side.cuda_stream, None), "default stream": (0, side)}[form]
    for _ in range(5):
        workspaces.clear()
        with torch.cuda.stream(current):
            got = calls(stream)
            # the current stream's next buffers are not those that the kernels work in
            assert len(workspaces) == 2 and all(size > 0 for _, size in workspaces)
            for size in [size for _, size in workspaces] * 2:
                other = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
                assert all(other.data_ptr() + size <= p or other.data_ptr() >= p + s for p, s in workspaces)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
