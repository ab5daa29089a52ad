"""Several answers to one prompt, decoded with drafted tokens, as a server would run it on one layer with experts.

    python examples/draft_decoding.py --answers 8 --prompt 700 --drafts 4 --steps 64

The prompt is taken in once and forked: the answers share its pages, and each gets a copy of the last one when it first grows.
A step drafts from each answer's own text (the token that followed last time), takes cache rows for the drafts, runs all of
them through the layer and the output head at once, lets the model's own distribution decide how many stand, and gives
the rows of the others back.  Lengths, tables and free pages live on the GPU and nothing waits for the host: the
whole step is one graph.  Weights are random, quantized on the GPU; normalisations and the text's table are torch's.
"""

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch
from decoder_layer import Layer, norm, rope_table

from ternary_bit_quantized_amd import q2_0 as B


class Server:
    """n_seqs answers of at most max_len tokens, `drafts` drafted tokens each a step, temperatures a list of one each."""

    def __init__(self, n_seqs, max_len, drafts, temperatures, vocab=1000, page=16, spare=8, groups=4, groups_used=2, seed=0, **layer):
        self.n, self.drafts, self.vocab, self.page, self.max_len = n_seqs, drafts, vocab, page, max_len
        self.layer = L = Layer(seed=seed, **layer)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.embed, self.head = (B.q2_0_quantize(torch.randn(vocab, L.hidden, generator=g, device="cuda")) for _ in range(2))
        self.bias = 0.05 * torch.randn(L.n_expert, generator=g, device="cuda")
        self.groups, self.groups_used = groups, groups_used
        cols = -(-max_len // page)
        n_pages = n_seqs * cols + spare
        self.k, self.v = (torch.zeros(n_pages, L.n_kv, page, L.head_dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.ref, self.free = B.q2_0_kv_pages(n_pages)
        ints = dict(dtype=torch.int32, device="cuda")
        self.table, self.lens = torch.full((n_seqs, cols), -1, **ints), torch.zeros(n_seqs, **ints)
        self.missing = torch.zeros(1, **ints)
        self.rope = rope_table(max_len, L.head_dim)
        self.temperature = torch.tensor(temperatures, dtype=torch.float32, device="cuda")
        self.cur = torch.zeros(n_seqs, **ints)                                # the last token of each, not in the cache yet
        self.follow = torch.full((n_seqs, vocab), -1, **ints)                 # what followed a token last time
        self.seq = torch.arange(n_seqs, **ints)

    def rows(self, ids):
        return norm(B.q2_0_get_rows(self.embed, self.vocab, self.layer.hidden, ids))

    def resize(self, new_lens):
        """(self.missing adds up: pages are reserved for max_len, so it stays 0)"""
        self.missing += B.q2_0_kv_resize(self.k, self.v, self.ref, self.free, self.table, self.lens, new_lens)

    def prompt(self, ids):
        """Takes in the prompt (int32 ids) but for its last token, and forks it to all answers."""
        n = ids.numel() - 1
        self.resize(torch.where(self.seq == 0, n, 0).int())
        _, k, v = self.layer.qkv(norm(self.rows(ids[:n])))
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        B.q2_0_kv_append(self.k, self.v, self.table, torch.zeros_like(pos), pos, k, v, rope=self.rope)
        B.q2_0_kv_fork(self.ref, self.table, self.page, self.lens, torch.zeros_like(self.seq[1:]), self.seq[1:])
        self.cur.copy_(ids[n:])
        # a token may stand in it many times: the last place counts
        last = torch.full((self.vocab,), -1, device="cuda").scatter_reduce_(0, ids[:n].long(), pos.long(), "amax")
        self.follow.copy_(torch.where(last >= 0, ids[last + 1], self.follow))

    def draft(self):
        """(tokens (n, drafts), how many of them): the answer's own text, as far as it goes on."""
        t, n_draft, known, out = self.cur, torch.zeros_like(self.cur), torch.ones_like(self.cur, dtype=torch.bool), []
        for _ in range(self.drafts):
            t = self.follow.gather(1, t.long().clamp(min=0)[:, None])[:, 0]
            known = known & (t >= 0)
            n_draft += known
            out.append(torch.where(known, t, 0))
        return torch.stack(out, 1) if out else self.follow[:, :0].contiguous(), n_draft

    def experts(self, x):
        L = self.layer
        logits = B.q2_0_mul_mat(L.router, L.n_expert, L.hidden, x, B.Q2_0_PREC_F32_MFMA)
        ids, weights = B.q2_0_moe_route_groups(logits, L.n_used, B.Q2_0_SCORE_SIGMOID, bias=self.bias, n_group=self.groups,
                                               n_group_used=self.groups_used, group_top=2, scale=2.0)
        parts = [slice(i, i + B.MOE_LAYER_MAX_TOKENS) for i in range(0, x.shape[0], B.MOE_LAYER_MAX_TOKENS)]
        return torch.cat([B.q2_0_moe_layer(L.gate, L.up, L.down, L.n_expert, L.n_ff, L.hidden, x[p], ids[p], weights[p])
                          for p in parts])

    def logits(self, ids):
        """Logits (n*(drafts+1), vocab) after each of the tokens ids (n, drafts+1), whose rows the cache takes."""
        L, nt = self.layer, self.drafts + 1
        first = self.lens.clone()
        self.resize(first + nt)
        h = self.rows(ids.flatten())
        q, k, v = L.qkv(norm(h))
        pos = (first[:, None] + torch.arange(nt, dtype=torch.int32, device="cuda")).flatten()
        rot = B.q2_0_kv_append(self.k, self.v, self.table, self.seq.repeat_interleave(nt), pos, k, v, rope=self.rope, q=q)
        att = B.q2_0_attn_shared(rot, self.k, self.v, self.table, self.lens, L.head_dim ** -0.5, max_len=self.max_len, n_qt=nt)
        mid = h + B.q2_0_mul_mat(L.wo, L.hidden, L.n_q * L.head_dim, att, B.Q2_0_PREC_F32_MFMA)
        out = mid + self.experts(norm(mid))
        return B.q2_0_mul_mat(self.head, self.vocab, L.hidden, norm(out), B.Q2_0_PREC_F32_MFMA) * 0.1

    def step(self, u, keep=None):
        """One step with the uniform numbers u (n, drafts + 1): (tokens (n, drafts + 1), -1 after the last; how many were drafted
        and stood).  keep: a dict that takes the stages' results."""
        tokens, n_draft = self.draft()
        first = self.lens.clone()
        logits = self.logits(torch.cat([self.cur[:, None], tokens], 1))
        out, taken = B.q2_0_draft_verify(logits, None, tokens, n_draft, u, temperature=self.temperature)
        self.resize(first + 1 + taken)
        # the text so far: what followed each token of this step, the last ones last
        before = torch.cat([self.cur[:, None], out[:, :-1]], 1)
        for j in range(self.drafts + 1):
            told = out[:, j: j + 1] >= 0
            at = before[:, j: j + 1].long().clamp(min=0)
            self.follow.scatter_(1, at, torch.where(told, out[:, j: j + 1], self.follow.gather(1, at)))
        self.cur.copy_(out.gather(1, taken.long()[:, None])[:, 0])
        if keep is not None:
            keep.update(tokens=tokens, n_draft=n_draft, first=first, logits=logits, out=out, taken=taken)
        return out, taken


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--answers", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    s = Server(a.answers, a.prompt + (a.steps + 4) * (a.drafts + 1), a.drafts, [0.0 if i % 2 else 0.7 for i in range(a.answers)])
    g = torch.Generator(device="cuda").manual_seed(2)
    s.prompt(torch.randint(0, s.vocab, (a.prompt,), generator=g, device="cuda", dtype=torch.int32))
    u = torch.rand(a.answers, a.drafts + 1, generator=g, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step(u)                                   # once outside the graph
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, taken = s.step(u)
    told = torch.zeros((), dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        u.uniform_(generator=g)
        graph.replay()
        told += (out >= 0).sum()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert int(s.missing) == 0 and int(out.max()) < s.vocab
    print("%d answers: %.1f us a step, %.2f tokens of each, %.0f tokens/s through the layer and head"
          % (a.answers, t / a.steps * 1e6, int(told) / a.steps / a.answers, int(told) / t))


if __name__ == "__main__":
    main()
