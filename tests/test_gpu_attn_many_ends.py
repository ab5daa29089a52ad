"""Many sequences that end at different places inside the shared prefix: their results, and that they cost no
more than one such sequence does (rows that see a whole key tile take it together, wherever they end)."""

import pytest
from test_gpu_attn_shared import check, shared_run

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,ct,page", [(64, "f16", 16), (128, "bf16", 24), (256, "bf16", 32)])
@pytest.mark.parametrize("n_q", [1, 4])
def test_results(dim, ct, page, n_q):
    lens = [13 * i + 1 for i in range(32)] + [420, 431]
    check(*shared_run(60, len(lens), 1, n_q, 1, dim, ct, page, 420, [12] * len(lens), lens=lens))


def test_time():
    import torch
    n, kv, dim, page, pre = 64, 8, 128, 64, 16384
    cols = pre // page + 1
    k, v = (torch.randn(cols, kv, page, dim, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(n, 4 * kv * dim, device="cuda").bfloat16()
    table = torch.arange(cols, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()

    def us(lens):
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        run = lambda: B.q2_0_attn_shared(q, k, v, table, ln, dim ** -0.5, prefix_len=pre)       # noqa: E731
        for _ in range(10):
            run()
        times = []
        for _ in range(9):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            for _ in range(10):
                run()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 100)
        return sorted(times)[4]

    full = pre + 30
    one = us([full] * 5 + [100] + [full] * (n - 6))
    many = us([pre * (i + 1) // 17 for i in range(15)] + [full] * (n - 15))
    print("one sequence ends inside the prefix %.1f us, fifteen at different places %.1f us" % (one, many))
    assert many < 1.4 * one
