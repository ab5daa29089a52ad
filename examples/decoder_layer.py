"""One decoder layer with experts, as a server would run it: a prompt that all sequences share is
taken in once, then the sequences decode together, one token each a step.

    python examples/decoder_layer.py --sequences 16 --prompt 1000 --steps 32

A step is seven library calls: q/k/v as one product group, the rotation with the cache append, attention
over the shared prompt and each sequence's own tokens, the output product, the router's product, the
choice of experts and the expert layer.  Weights are random, quantized on the GPU; the
normalisations between are torch's.  The decode step is captured in a graph once and replayed:
positions and lengths live on the GPU and advance inside it.
"""

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from ternary_bit_quantized_amd import q2_0 as B


class Layer:
    """Q2_0 weights of a layer: attention with n_q query and n_kv key heads of head_dim, n_expert experts of
    n_ff, of which a token uses n_used."""

    def __init__(self, hidden=2048, n_q=32, n_kv=4, head_dim=128, n_expert=128, n_ff=768, n_used=8, seed=0):
        self.hidden, self.n_q, self.n_kv, self.head_dim = hidden, n_q, n_kv, head_dim
        self.n_expert, self.n_ff, self.n_used = n_expert, n_ff, n_used
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return B.q2_0_quantize(torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5)

        self.wq, self.wk, self.wv = (weight(n * head_dim, hidden) for n in (n_q, n_kv, n_kv))
        self.wo = weight(hidden, n_q * head_dim)
        self.router = weight(n_expert, hidden)
        # the experts' matrices back to back
        self.gate, self.up = (weight(n_expert * n_ff, hidden) for _ in range(2))
        self.down = weight(n_expert * hidden, n_ff)

    def qkv(self, x, precision=B.Q2_0_PREC_F32_MFMA):
        n = self.head_dim
        return B.q2_0_mul_mat_group([(self.wq, self.n_q * n), (self.wk, self.n_kv * n), (self.wv, self.n_kv * n)], self.hidden, x,
                                    precision)

    def experts(self, x):
        logits = B.q2_0_mul_mat(self.router, self.n_expert, self.hidden, x, B.Q2_0_PREC_F32_MFMA)
        ids, weights = B.q2_0_moe_route(logits, self.n_used)
        return ids, weights, B.q2_0_moe_layer(self.gate, self.up, self.down, self.n_expert, self.n_ff, self.hidden, x, ids, weights)


class Cache:
    """A paged cache for n_seqs sequences that share their first prefix tokens: the prefix's whole pages stand in
    every row of the table, its last page (where it ends inside one) has a copy per sequence, and each
    sequence has pages for own_max tokens more."""

    def __init__(self, layer, n_seqs, prefix, own_max, page=64, dtype=torch.bfloat16):
        cols, shared = -(-(prefix + own_max) // page), prefix // page
        n_pages = shared + n_seqs * (cols - shared)
        self.k, self.v = (torch.zeros(n_pages, layer.n_kv, page, layer.head_dim, dtype=dtype, device="cuda") for _ in range(2))
        own = shared + torch.arange(n_seqs * (cols - shared), device="cuda").view(n_seqs, -1)
        self.table = torch.cat([torch.arange(shared, device="cuda").expand(n_seqs, -1), own], 1).to(torch.int32).contiguous()
        self.n_seqs, self.prefix, self.max_len, self.page = n_seqs, prefix, prefix + own_max, page

    def share_last_page(self):
        """Copies the page in which the prefix ends from the first sequence to the others."""
        if self.prefix % self.page:
            at = self.table[:, self.prefix // self.page].long()
            for pool in (self.k, self.v):
                pool[at[1:]] = pool[at[:1]].clone()


def rope_table(n_pos, rot_dim, base=10000.0):
    """(n_pos, rot_dim) float32: cos then sin of each position's angles, worked out in 64 bits."""
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def norm(x):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)


def prompt(layer, cache, rope, h):
    """Puts the shared prompt's keys and values in the cache (h: its prefix rows of the hidden state)."""
    n = h.shape[0]
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    _, k, v = layer.qkv(norm(h))
    B.q2_0_kv_append(cache.k, cache.v, cache.table, seq, pos, k, v, rope=rope)
    cache.share_last_page()


def step(layer, cache, rope, h, seq, lens, keep=None):
    """One token of every sequence: h (n_seqs, hidden) -> the layer's output; lens (tokens so far) grows by one.
    keep: a dict that takes the stages' results."""
    x = norm(h)
    q, k, v = layer.qkv(x)
    rot = B.q2_0_kv_append(cache.k, cache.v, cache.table, seq, lens, k, v, rope=rope, q=q)
    lens.add_(1)
    att = B.q2_0_attn_shared(rot, cache.k, cache.v, cache.table, lens, layer.head_dim ** -0.5, prefix_len=cache.prefix,
                             max_len=cache.max_len)
    mid = h + B.q2_0_mul_mat(layer.wo, layer.hidden, layer.n_q * layer.head_dim, att, B.Q2_0_PREC_F32_MFMA)
    y = norm(mid)
    ids, weights, moe = layer.experts(y)
    if keep is not None:
        keep.update(x=x, q=q, k=k, v=v, rot=rot, att=att, mid=mid, y=y, ids=ids, weights=weights, moe=moe)
    return mid + moe


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--sequences", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    layer = Layer()
    cache = Cache(layer, a.sequences, a.prompt, a.steps + 8)
    rope = rope_table(cache.max_len, layer.head_dim)
    g = torch.Generator(device="cuda").manual_seed(1)
    if a.prompt:
        prompt(layer, cache, rope, torch.randn(a.prompt, layer.hidden, generator=g, device="cuda"))
    h = torch.randn(a.sequences, layer.hidden, generator=g, device="cuda")
    seq = torch.arange(a.sequences, dtype=torch.int32, device="cuda")
    lens = torch.full((a.sequences,), a.prompt, dtype=torch.int32, device="cuda")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                   # once outside the graph; its token is written again below
        step(layer, cache, rope, h, seq, lens)
        lens.sub_(1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(layer, cache, rope, h, seq, lens)
        h.copy_(out)                                # (a model would sample a token and embed it here)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, a.steps)
    assert torch.isfinite(h).all() and (lens == a.prompt + a.steps).all()
    print("%d sequences, prompt of %d shared: %.1f us a step, %.0f tokens/s through the layer"
          % (a.sequences, a.prompt, t * 1e6, a.sequences / t))


if __name__ == "__main__":
    main()
