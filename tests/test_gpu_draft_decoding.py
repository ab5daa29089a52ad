"""The example that decodes with drafted tokens: its stages against their definitions, its text against decoding one
token at a time, its cache against the text, its pages against each other, and its step in a graph."""

import importlib.util
import os
import sys

import numpy as np
import pytest
from test_gpu_draft_verify import reference as verified

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(vocab=300, page=16, hidden=192, n_q=4, n_kv=2, head_dim=64, n_expert=16, n_ff=128, n_used=3)


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    spec = importlib.util.spec_from_file_location("draft_decoding", os.path.join(ROOT, "examples", "draft_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def server(E, n, drafts, temperatures, prompt=37, seed=0):
    import torch
    s = E.Server(n, 200, drafts, temperatures, seed=seed, **SIZES)
    g = torch.Generator(device="cuda").manual_seed(seed + 7)
    ids = torch.randint(0, s.vocab, (prompt,), generator=g, device="cuda", dtype=torch.int32)
    ids[prompt // 2:] = ids[: prompt - prompt // 2].clone()       # a text that repeats itself
    s.prompt(ids)
    return s, ids, g


def pages_add_up(s):
    """Every page is held as often as it stands in a row, and is free if it never does."""
    counts = [0] * s.ref.numel()
    for row, n in zip(s.table.tolist(), s.lens.tolist()):
        held = -(-n // s.page)
        for p in row[:held]:
            counts[p] += 1
        assert all(p == -1 for p in row[held:])
    assert counts == s.ref.tolist()
    words = [w & 0xFFFFFFFF for w in s.free.tolist()]
    assert [words[i // 32] >> (i % 32) & 1 for i in range(len(counts))] == [int(c == 0) for c in counts]
    assert int(s.missing) == 0


@pytest.mark.parametrize("n,drafts", [(1, 0), (3, 4), (6, 15), (20, 2)])
def test_steps(n, drafts):
    import torch
    E = example()
    s, ids, g = server(E, n, drafts, [[0.0, 0.8, 1.3][i % 3] for i in range(n)])
    texts = [ids.tolist() for _ in range(n)]
    assert s.lens.tolist() == [len(ids) - 1] * n and (n == 1 or int(s.ref.max()) == n)
    pages_add_up(s)
    took = 0
    for _ in range(6):
        u = torch.rand(n, drafts + 1, generator=g, device="cuda")
        keep = {}
        out, taken = s.step(u, keep)
        torch.cuda.synchronize()
        pages_add_up(s)
        want, number = verified(keep["logits"].double().cpu().numpy(), None, keep["tokens"].cpu().numpy(),
                                keep["n_draft"].cpu().numpy(), u.double().cpu().numpy(), temp=s.temperature.double().cpu().numpy())
        assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(taken.cpu().numpy(), number)
        for t, o, a in zip(texts, out.tolist(), taken.tolist()):
            t += o[: a + 1]
            took += a
        assert s.lens.tolist() == [len(t) - 1 for t in texts] and s.cur.tolist() == [t[-1] for t in texts]
    assert took > 0 or drafts == 0
    # the cache holds the keys of the text, each answer's own, whatever was drafted and refused in between
    from ternary_bit_quantized_amd import q2_0 as B
    for i, t in enumerate(texts):
        m = len(t) - 1
        _, k, v = s.layer.qkv(E.norm(s.rows(torch.tensor(t[:m], dtype=torch.int32, device="cuda"))))
        pos = torch.arange(m, dtype=torch.int32, device="cuda")
        kc, vc = torch.zeros_like(s.k), torch.zeros_like(s.v)
        B.q2_0_kv_append(kc, vc, s.table, torch.full_like(pos, i), pos, k, v, rope=s.rope)
        where, row = s.table[i][(pos // s.page).long()].long(), (pos % s.page).long()
        for pool, again in ((s.k, kc), (s.v, vc)):
            a, b = pool[where, :, row].float(), again[where, :, row].float()
            # two products of 1e-5 * sum |W x| each, a turn, and a rounding of 2^-8 on either side: elements of some units
            assert torch.all((a - b).abs() <= 2 * 2.0 ** -8 * b.abs() + 1e-2)


def test_greedy_text_is_that_of_one_token_at_a_time():
    import torch
    E = example()
    texts, gaps, took = {}, [[], []], 0
    for d in (0, 5):
        s, _, _ = server(E, 2, d, [0.0, 0.0], seed=3)
        s.cur[1] = 5                            # two answers that differ
        got = [[], []]
        while min(len(t) for t in got) < 40:
            keep = {}
            out, taken = s.step(torch.zeros(2, d + 1, device="cuda"), keep)
            for i in range(2):
                got[i] += out[i, : int(taken[i]) + 1].tolist()
                if d == 0:
                    top = keep["logits"][i].topk(2).values
                    gaps[i].append(float(top[0] - top[1]))
            took += int(taken.sum())
        texts[d] = got
    assert took > 0
    for i in range(2):
        # the same text up to where two logits are so close that the rounding of keys and values to bfloat16 may decide
        sure = next((j for j, gap in enumerate(gaps[i]) if gap < 0.05), 40)
        assert sure > 0 and texts[0][i][:sure] == texts[5][i][:sure]


def test_captured_step():
    import torch
    E = example()
    n, drafts = 5, 4
    temps = [0.0, 0.7, 1.0, 1.3, 0.0]
    g = torch.Generator(device="cuda").manual_seed(1)
    us = [torch.rand(n, drafts + 1, generator=g, device="cuda") for _ in range(8)]
    eager, _, _ = server(E, n, drafts, temps, seed=4)
    want = [[t.clone() for t in eager.step(u)] + [eager.lens.clone(), eager.table.clone(), eager.free.clone()] for u in us]
    s, _, _ = server(E, n, drafts, temps, seed=4)
    u = us[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in s.step(u)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, taken = s.step(u)
    for i in range(1, len(us)):
        u.copy_(us[i])
        graph.replay()
        torch.randn(300, 300, device="cuda").sum().item()         # the program's own work in between
        assert all(torch.equal(a, b) for a, b in zip((out, taken, s.lens, s.table, s.free), want[i])), i
    pages_add_up(s)

def test_a_prompt_that_goes_on_differently():
    """Drafts come from what followed a token last in the prompt, however often it stands there."""
    import torch
    E = example()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = torch.randint(0, [2, 7, 40, 300][seed], (190,), generator=g, device="cuda", dtype=torch.int32)
        s = E.Server(3, 200, 2, [0.0] * 3, seed=seed, **SIZES)
        s.prompt(ids)
        text, want = ids.tolist(), [-1] * s.vocab
        for a, b in zip(text, text[1:]):
            want[a] = b
        assert s.follow.tolist() == [want] * 3


def test_example_runs(monkeypatch, capsys):
    E = example()
    monkeypatch.setattr(sys, "argv", ["draft_decoding.py", "--answers", "3", "--prompt", "50", "--drafts", "3", "--steps", "5"])
    E.main()
    assert "tokens/s" in capsys.readouterr().out
