"""The operators between two decoder steps on streams that are not the current one, captured in graphs and replayed, and two
calls at once."""

import pytest
from test_gpu_draft_verify import case
from test_gpu_kv_pages import Both, pool

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu


class Call:
    """Inputs that can be set, and a call that returns its results (or the buffers that it changes)."""

    def __init__(self, name, seed):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.name = name
        if name == "route":
            self.inputs = [torch.randn(300, 128, generator=g, device="cuda")]
        elif name in ("verify", "probs"):
            self.form = B.Q2_0_DRAFT_PROBS if name == "probs" else B.Q2_0_DRAFT_LOGITS
            self.inputs = list(case(9, 3, 20011, form="probs" if name == "probs" else "logits", seed=seed))
        elif name == "copy":
            self.inputs = pool(8, 2, 16, 64, "heads", seed, torch.float16) + pool(8, 2, 16, 64, "tokens", seed + 1, torch.float16)
            self.inputs += [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([seed % 8, 3], [1, 6])]
        elif name == "compact":
            free = torch.tensor([0x0F0F5A00 + seed], dtype=torch.int32, device="cuda")
            table = torch.randint(0, 30, (3, 4), generator=g, device="cuda", dtype=torch.int32)
            self.inputs = pool(30, 2, 16, 64, "heads", seed, torch.float16) + pool(28, 2, 16, 64, "heads", seed + 1, torch.float16)
            self.inputs += [torch.arange(30, dtype=torch.int32, device="cuda"), free, table,
                            torch.tensor([3, 64, 40], dtype=torch.int32, device="cuda"), torch.zeros(28, dtype=torch.int32, device="cuda"),
                            torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(3, 4, dtype=torch.int32, device="cuda")]
        else:       # resize, fork, resize: a shared page becomes two
            t = Both(n_pages=64 + 3000 * (name == "large steps"), n_seqs=6 + 90 * (name == "large steps"),
                     cols=9 + 991 * (name == "large steps"), seed=seed)
            n = t.m.n_seqs
            t.resize([20 + seed % 5] + [0] * (n - 3) + [100, 40])
            t.m = None
            self.inputs = [t.k, t.v, t.ref, t.free, t.table, t.lens] + \
                [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 0], [1, 2], [22] * 3 + [-1] * (n - 4) + [70])]

    def __call__(self, stream=None):
        i = self.inputs
        if self.name == "route":
            return list(B.q2_0_moe_route_groups(i[0], 6, n_group=8, n_group_used=3, group_top=2, stream=stream))
        if self.name in ("verify", "probs"):
            return list(B.q2_0_draft_verify(*i, form=self.form, stream=stream))
        if self.name == "copy":
            B.q2_0_kv_copy(i[0], i[1], i[2], i[3], i[4], i[5], stream=stream)
            return i[:2]
        if self.name == "compact":
            n = B.q2_0_kv_compact(i[2], i[3], i[8], i[9], i[10], i[0], i[1], i[4], i[5], i[6], i[7], stream=stream)
            return i[2:4] + i[8:11] + [n]
        B.q2_0_kv_fork(i[2], i[4], 16, i[5], i[6], i[7], stream=stream)
        n = B.q2_0_kv_resize(*i[:6], i[8], stream=stream)
        return i[:6] + [n]


NAMES = ["route", "verify", "probs", "copy", "compact", "steps", "large steps"]


def results(name, seed, stream=None):
    import torch
    got = [t.clone() for t in Call(name, seed)(stream)]
    torch.cuda.synchronize()
    return got


def same(a, b):
    import torch
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("handle", [False, True])
def test_another_stream(name, handle):
    import torch
    want = results(name, 1)
    side = torch.cuda.Stream()
    for _ in range(3):
        c = Call(name, 1)
        torch.cuda.synchronize()
        got = c(side.cuda_stream if handle else side)
        # the current stream's next buffers are none of the call's
        for size in (64, 512, 4096, 100000):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_two_at_once(name):
    import torch
    want = [results(name, s) for s in (1, 2)]
    for _ in range(3):
        calls = [Call(name, s) for s in (1, 2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = [c(s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        same(got[0], want[0])
        same(got[1], want[1])


@pytest.mark.parametrize("name", NAMES)
def test_replays(name):
    import torch
    sets = [Call(name, s).inputs for s in (1, 2, 3)]
    want = [results(name, s) for s in (1, 2, 3)]
    c = Call(name, 1)
    with torch.cuda.stream(torch.cuda.Stream()):
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c()
    for turn in range(6):
        for buf, v in zip(c.inputs, sets[turn % 3]):
            if buf is not None:
                buf.copy_(v)
        for t in out:
            if not any(t is i for i in c.inputs):
                t.fill_(-77)
        graph.replay()
        a = torch.randn(256, 256, device="cuda")
        float((a @ a).sum())                    # the program's own work, and a synchronization
        same(out, want[turn % 3])
