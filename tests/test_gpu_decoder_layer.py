"""The example's decoder layer: every stage of a step against its definition in 64 bits on the values that the
stage before it left, and the captured step against the eager one."""

import importlib.util
import os

import numpy as np
import pytest

import oracle
from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
REL = 1e-5                       # a product's contract: 1e-5 * sum |W x|
U = 2.0 ** -8                    # bfloat16


def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def host(t):
    return t.detach().double().cpu().numpy()


def product(w, M, K, x):
    return oracle.mul_mat(w.cpu().numpy().reshape(-1), M, K, np.ascontiguousarray(x, dtype=np.float32))


def near(got, ref, tol, what):
    err = np.abs(host(got) - ref)
    assert np.all(err <= tol), "%s: worst %.3g of its tolerance" % (what, np.max(err / tol))


def setup(E, seqs, prefix, own):
    import torch
    layer = E.Layer(hidden=192, n_q=4, n_kv=2, head_dim=64, n_expert=10, n_ff=128, n_used=3, seed=3)
    cache = E.Cache(layer, seqs, prefix, own, page=16)
    rope = E.rope_table(cache.max_len, layer.head_dim)
    g = torch.Generator(device="cuda").manual_seed(4)
    if prefix:
        E.prompt(layer, cache, rope, torch.randn(prefix, layer.hidden, generator=g, device="cuda"))
    h = torch.randn(seqs, layer.hidden, generator=g, device="cuda")
    seq = torch.arange(seqs, dtype=torch.int32, device="cuda")
    lens = torch.full((seqs,), prefix, dtype=torch.int32, device="cuda")
    return layer, cache, rope, h, seq, lens


@pytest.mark.parametrize("seqs,prefix", [(1, 0), (3, 40), (12, 33)])
def test_stages(seqs, prefix):
    E = example()
    layer, cache, rope, h, seq, lens = setup(E, seqs, prefix, 8)
    H, D = layer.hidden, layer.head_dim
    for n in range(3):
        keep = {}
        out = E.step(layer, cache, rope, h, seq, lens, keep)
        length = prefix + n + 1
        assert lens.tolist() == [length] * seqs
        for name, w, heads in (("q", layer.wq, layer.n_q), ("k", layer.wk, layer.n_kv), ("v", layer.wv, layer.n_kv)):
            ref, size = product(w, heads * D, H, host(keep["x"]))
            near(keep[name], ref, REL * size + 1e-30, name)
        # rotation and cache: two products and a sum in f32, one rounding
        table = host(rope)[length - 1]
        c, s = table[: D // 2], table[D // 2:]
        place = cache.table.cpu().numpy()[:, (length - 1) // 16], (length - 1) % 16

        def turn(t):
            a = host(t).reshape(seqs, -1, D)
            x, y = a[..., : D // 2], a[..., D // 2:]
            ref = np.concatenate([x * c - y * s, y * c + x * s], -1)
            size = np.concatenate([abs(x * c) + abs(y * s), abs(y * c) + abs(x * s)], -1)
            return ref, U * abs(ref) + 3 * 2.0 ** -24 * (1 + U) * size + 2.0 ** -25

        ref, tol = turn(keep["q"])
        near(keep["rot"].view(seqs, -1, D), ref, tol, "rotated q")
        ref, tol = turn(keep["k"])
        near(cache.k[place[0].tolist(), :, place[1]], ref, tol, "cached k")
        ref = host(keep["v"]).reshape(seqs, -1, D)
        near(cache.v[place[0].tolist(), :, place[1]], ref, U * abs(ref) + 2.0 ** -25, "cached v")
        # attention over what the cache holds
        kc, vc, tab = host(cache.k), host(cache.v), cache.table.cpu().numpy()
        i = np.arange(length)
        for b in range(seqs):
            ks, vs = (a[tab[b][i // 16], :, i % 16].transpose(1, 0, 2) for a in (kc, vc))
            x = host(keep["rot"])[b].reshape(layer.n_kv, -1, D)
            sc = D ** -0.5 * (x @ ks.transpose(0, 2, 1))
            size = D ** -0.5 * (abs(x) @ abs(ks).transpose(0, 2, 1)).max(2, keepdims=True)
            p = np.exp(sc - sc.max(2, keepdims=True))
            p /= p.sum(2, keepdims=True)
            delta = (D + 4 + length) * 2.0 ** -24 * (size + 1)
            ref = p @ vs
            near(keep["att"][b].view(layer.n_kv, -1, D), ref, (U + 2 * delta) * (p @ abs(vs)) + U * abs(ref) + 2.0 ** -24, "attention")
        ref, size = product(layer.wo, H, layer.n_q * D, host(keep["att"]))
        near(keep["mid"], ref + host(h), REL * size + 2.0 ** -23 * (abs(ref) + abs(host(h))), "output product")
        # the chosen experts are the largest logits but for the product's error
        y = host(keep["y"])
        logits, size = product(layer.router, layer.n_expert, H, y)
        ids = keep["ids"].cpu().numpy()
        for b in range(seqs):
            least = logits[b][ids[b]].min()
            rest = np.delete(logits[b], ids[b])
            assert len(set(ids[b])) == layer.n_used and least >= rest.max() - 2 * REL * size[b].max()
            w = np.exp(logits[b][ids[b]] - logits[b].max())
            near(keep["weights"][b], w / w.sum(), 4 * REL * size[b].max() + 1e-5, "weights")
        # the expert layer on the ids and weights given
        F = layer.n_ff
        mats = [m.cpu().numpy().reshape(layer.n_expert, -1) for m in (layer.gate, layer.up, layer.down)]
        for b in range(seqs):
            ref, tol = np.zeros(H), np.zeros(H)
            for u, e in enumerate(ids[b]):
                xb = np.ascontiguousarray(y[b:b + 1], dtype=np.float32)
                (gv, ga), (uv, ua) = ([r[0] for r in oracle.mul_mat(m[e], F, H, xb)] for m in mats[:2])
                s = gv / (1 + np.exp(-gv))
                hid = s * uv
                dh = 1.1 * REL * ga * abs(uv) + REL * ua * abs(s) + 2.0 ** -23 * (5 + abs(gv)) * abs(hid)
                z, za = (r[0] for r in oracle.mul_mat(mats[2][e], H, F, hid.astype(np.float32)[None]))
                dz = oracle.mul_mat(mats[2][e], H, F, dh.astype(np.float32)[None])[1][0]
                wt = float(keep["weights"][b, u])
                ref += wt * z
                tol += wt * (REL * za + dz) + 2.0 ** -23 * layer.n_used * wt * abs(z)
            near(keep["moe"][b], ref, tol * 1.001 + 1e-30, "expert layer")
        h = out


@pytest.mark.parametrize("seqs,prefix", [(3, 40), (40, 200)])
def test_captured_step(seqs, prefix):
    """Replays of the captured step, other work and eager steps between them, give bit for bit the eager results."""
    import torch
    E = example()
    layer, cache, rope, h, seq, lens = setup(E, seqs, prefix, 12)
    start, k0, v0 = h.clone(), cache.k.clone(), cache.v.clone()

    def reset():
        h.copy_(start), cache.k.copy_(k0), cache.v.copy_(v0), lens.fill_(prefix)

    eager = []
    for _ in range(4):
        h.copy_(E.step(layer, cache, rope, h, seq, lens))
        eager.append(h.clone())
    k1, v1 = cache.k.clone(), cache.v.clone()
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.copy_(E.step(layer, cache, rope, h, seq, lens))
    for again in range(2):
        reset()
        for want in eager:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, want)
            junk = torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")
            B.q2_0_moe_route(junk[:, :10], 3)
            torch.cuda.synchronize()
        assert torch.equal(cache.k, k1) and torch.equal(cache.v, v1)
