"""Pages of the cache -- copies, forks, growing and shrinking sequences, a move into another pool -- against a model that
does them one page at a time.  Everything is whole numbers and copied bits, so all of it has to be the same."""

import random

import numpy as np
import pytest

from ternary_bit_quantized_amd import q2_0 as B

pytestmark = pytest.mark.gpu


def pages_of(n, page):
    return -(-n // page)


class Model:
    """The state of a pool on the host: pools as bit patterns (pages, heads, rows, dim)."""

    def __init__(self, n_pages, n_seqs, cols, page):
        self.n_pages, self.n_seqs, self.cols, self.page = n_pages, n_seqs, cols, page
        self.ref, self.free = [0] * n_pages, set(range(n_pages))
        self.table = [[-1] * cols for _ in range(n_seqs)]
        self.lens = [0] * n_seqs
        self.k = self.v = None

    def good(self, n):
        return 0 <= n <= self.cols * self.page

    def resize(self, new):
        page, ok = self.page, [self.good(a) and self.good(b) for a, b in zip(self.lens, new)]
        for s in range(self.n_seqs):
            if ok[s] and new[s] < self.lens[s]:
                for i in range(pages_of(new[s], page), pages_of(self.lens[s], page)):
                    p, self.table[s][i] = self.table[s][i], -1
                    if 0 <= p < self.n_pages:
                        self.ref[p] -= 1
                        if self.ref[p] == 0:
                            self.free.add(p)
                self.lens[s] = new[s]
        grow = [s for s in range(self.n_seqs) if ok[s] and new[s] > self.lens[s]]
        held = {}
        for s in grow:
            if self.lens[s] % page:
                p = self.table[s][self.lens[s] // page]
                if 0 <= p < self.n_pages and self.ref[p] > 1:
                    held.setdefault(p, []).append(s)
        copied = {s for p, who in held.items() for s in (who[1:] if len(who) == self.ref[p] else who)}
        need = sum(pages_of(new[s], page) - pages_of(self.lens[s], page) + (s in copied) for s in grow)
        if need > len(self.free):
            return need - len(self.free)
        take = iter(sorted(self.free)[:need])
        for s in grow:
            if s in copied:
                i, p = self.lens[s] // page, next(take)
                old, self.table[s][i] = self.table[s][i], p
                for pool in (self.k, self.v):
                    pool[p, :, : self.lens[s] % page] = pool[old, :, : self.lens[s] % page]
                self.ref[old] -= 1
                self.ref[p] = 1
                self.free.remove(p)
            for i in range(pages_of(self.lens[s], page), pages_of(new[s], page)):
                p = self.table[s][i] = next(take)
                self.ref[p] = 1
                self.free.remove(p)
            self.lens[s] = new[s]
        return 0

    def fork(self, src, dst):
        lens = list(self.lens)
        taken = set()
        for a, b in zip(src, dst):
            if not (0 <= a < self.n_seqs and 0 <= b < self.n_seqs) or a == b or lens[b] != 0 or b in taken or not self.good(lens[a]):
                continue
            taken.add(b)
            for i in range(pages_of(lens[a], self.page)):
                p = self.table[b][i] = self.table[a][i]
                if 0 <= p < self.n_pages:
                    self.ref[p] += 1
            self.lens[b] = lens[a]


def words(free, n):
    w = [0] * ((n + 31) // 32)
    for i in free:
        w[i // 32] |= 1 << (i % 32)
    return np.array(w, np.uint32).view(np.int32)


class Both:
    """A model and the device's state, changed together and compared after each call."""

    def __init__(self, n_pages=70, n_seqs=5, cols=9, page=16, n_kv=2, dim=64, dtype="bf16", layout="heads", seed=0, pad_cols=0):
        import torch
        self.m = Model(n_pages, n_seqs, cols, page)
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
        if layout == "heads":
            self.k, self.v = (torch.randn(n_pages, n_kv, page, dim, generator=g, device="cuda").to(dt) for _ in range(2))
        elif layout == "tokens":
            self.k, self.v = (torch.randn(n_pages, page, n_kv, dim, generator=g, device="cuda").to(dt).transpose(1, 2)
                              for _ in range(2))
        else:       # keys and values of a token side by side, with a gap
            both = torch.randn(n_pages, n_kv, page, 2 * dim + 8, generator=g, device="cuda").to(dt)
            self.k, self.v = both[..., :dim], both[..., dim: 2 * dim]
        self.m.k, self.m.v = self.bits(self.k), self.bits(self.v)
        self.ref, self.free = B.q2_0_kv_pages(n_pages)
        self.table = torch.full((n_seqs, cols + pad_cols), -1, dtype=torch.int32, device="cuda")[:, :cols]
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")

    @staticmethod
    def bits(t):
        import torch
        return t.contiguous().view(torch.int16).cpu().numpy().copy()

    def ints(self, v):
        import torch
        return torch.tensor(np.asarray(v, np.int32), device="cuda")

    def same(self, what=""):
        import torch
        torch.cuda.synchronize()
        m = self.m
        assert self.lens.tolist() == m.lens, what
        assert self.table.tolist() == m.table, what
        assert self.ref.tolist() == m.ref, what
        n = m.n_pages
        mask = words(range(n), n)
        assert np.array_equal(self.free.cpu().numpy() & mask, words(m.free, n)), what
        assert np.array_equal(self.bits(self.k), m.k) and np.array_equal(self.bits(self.v), m.v), what

    def resize(self, new, **kw):
        missing = B.q2_0_kv_resize(self.k, self.v, self.ref, self.free, self.table, self.lens, self.ints(new), **kw)
        want = self.m.resize(list(new))
        self.same("resize to %s" % (new,))
        assert missing.item() == want
        return want

    def fork(self, src, dst):
        B.q2_0_kv_fork(self.ref, self.table, self.m.page, self.lens, self.ints(src), self.ints(dst))
        self.m.fork(src, dst)
        self.same("fork %s to %s" % (src, dst))


@pytest.mark.parametrize("layout", ["heads", "tokens", "beside"])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "f16"), (256, "bf16")])
def test_a_life_of_sequences(layout, dim, dtype):
    t = Both(dim=dim, dtype=dtype, layout=layout, seed=dim)
    t.resize([17, 0, 16, 1, 144])
    t.resize([17, 5, 16, 0, 144])
    t.resize([18, 5, 33, -1, 100])
    t.fork([0, 4], [3, 1])                   # (1 is not empty)
    t.resize([-1, 0, -1, -1, -1])
    t.fork([4], [1])
    t.resize([30, 101, 33, 19, 101])         # both holders of each shared last page grow
    t.resize([0] * 5)
    assert t.m.free == set(range(70))
    t.resize([144] * 5)


@pytest.mark.parametrize("page", [1, 3, 16, 20, 1000])
def test_page_sizes(page):
    t = Both(n_pages=40, cols=7, page=page, n_kv=1, seed=page)
    t.resize([page, page + 1, 2 * page - 1, 3 * page, 7 * page])
    t.resize([0, page, 5 * page, -1, 2 * page + 1])
    t.fork([2], [0])
    t.resize([5 * page + 1, page + 1, 5 * page + 1, -1, 0])
    t.fork([0, 3], [4, 4])
    t.resize([6 * page, 1, 6 * page, 3 * page + 2, 7 * page])


def test_shared_last_pages():
    t = Both(n_pages=64, n_seqs=8, cols=5, page=16)
    t.resize([20, 0, 0, 0, 33, 0, 0, 0])
    t.fork([0, 0, 0, 4], [1, 2, 3, 5])
    t.resize([-1, 21, -1, -1, -1, -1, -1, -1])                # one of four: a copy, three go on sharing
    t.resize([21, -1, 22, 23, -1, -1, -1, -1])                # the three that are left: the first keeps the page
    t.resize([16, 16, 16, 16, 33, 40, 0, 0])                  # back to whole shared pages, which nothing copies
    t.fork([4, 4], [6, 7])
    t.resize([17, 17, 17, 17, -1, -1, 0, 64])
    t.resize([10, 10, 10, 10, 8, 8, 8, 8])                    # into the middle of shared pages
    t.resize([11, 12, 13, 14, 9, 9, 9, 9])
    # a holder that leaves in the same call: the other has the page to itself
    t.resize([0] * 8)
    t.resize([8, 0, 0, 0, 0, 0, 0, 0])
    t.fork([0, 0], [1, 2])
    t.resize([0, 9, 0, -1, -1, -1, -1, -1])
    assert len(t.m.free) == 63
    # held by an owner outside the table: never given away
    t.ref[t.m.table[1][0]] += 1
    t.m.ref[t.m.table[1][0]] += 1
    t.resize([0, 10, 0, 0, 0, 0, 0, 0])
    assert len(t.m.free) == 62


def test_too_few_pages():
    t = Both(n_pages=10, n_seqs=4, cols=9, page=4)
    assert t.resize([36, 5, 0, 0]) == 1
    assert t.resize([36, 4, 0, 0]) == 0
    assert t.resize([37, 4, 0, 0]) == 0                       # (37 is beyond the row: left)
    t.resize([30, 4, 0, 0])
    t.fork([0], [2])
    assert t.resize([31, 5, 31, -1]) == 1                     # a copy and a page, one is free
    assert t.resize([31, -1, 31, -1]) == 0
    assert t.resize([0, 36, 36, 36]) == 17                    # 8 + 1 + 9, one is free: what shrinks does so all the same
    assert t.resize([36, 0, 0, 0]) == 0
    assert t.resize([0, 0, 0, 36]) == 0                       # pages that one leaves another takes


def test_lengths_and_pages_that_do_not_exist():
    t = Both(n_pages=33, n_seqs=6, cols=4, page=16, pad_cols=3)
    t.resize([64, 65, -1, 2 ** 31 - 1, -(2 ** 31), 20])
    for s, p in ((0, 33), (5, -7)):
        i = t.m.lens[s] // 16 - (s == 0)
        t.table[s, i] = t.m.table[s][i] = p
    t.resize([40, 0, 0, 0, 0, 21])
    t.resize([0, 10, 10, 10, 10, 0])
    t.lens[2] = t.m.lens[2] = -3
    t.lens[3] = t.m.lens[3] = 65
    t.resize([1, 0, 5, 5, 5, 5])
    t.fork([2, 3, 4, 4, -1, 9, 4, 4], [1, 1, 4, 9, 1, 1, -2, 1])
    t.resize([0, -1, -1, -1, -1, -1])


def test_forks():
    t = Both(n_seqs=9)
    t.resize([30, 0, 0, 144, 0, 0, 0, 0, 0])
    t.fork([0, 3, 0, 1, 3], [1, 1, 2, 4, 3])                  # one destination twice, an empty parent, itself
    t.fork([1, 2], [5, 6])                                    # of forks
    t.fork([], [])
    assert t.m.lens == [30, 30, 30, 144, 0, 30, 30, 0, 0]
    t.fork([7, 3], [8, 7])                                    # 7 is empty before the call: so is its fork
    assert t.m.lens[7:] == [144, 0]


def test_a_pool_at_random():
    r = random.Random(5)
    for n_pages, page in ((31, 4), (64, 5), (200, 2)):
        n = 12
        t = Both(n_pages=n_pages, n_seqs=n, cols=8, page=page, n_kv=1, seed=n_pages)
        for _ in range(25):
            new = [r.choice([-1, -1, 0, t.m.lens[s], t.m.lens[s] + 1, r.randint(0, 8 * page), max(0, t.m.lens[s] - 2)])
                   for s in range(n)]
            t.resize(new)
            t.fork([r.randint(0, n - 1) for _ in range(4)], [r.randint(0, n - 1) for _ in range(4)])
        counts = [0] * n_pages
        for s in range(n):
            for i in range(pages_of(t.m.lens[s], page)):
                counts[t.m.table[s][i]] += 1
        assert counts == t.m.ref and t.m.free == {p for p in range(n_pages) if counts[p] == 0}


@pytest.mark.parametrize("n_seqs,cols", [(1, 3000), (1024, 3), (1025, 2), (8192, 2), (300, 1100), (2000, 50)])
def test_many_sequences_and_long_rows(n_seqs, cols):
    import torch
    page, n_pages = 4, min(400000, n_seqs * cols + 77)
    t = Both(n_pages=n_pages, n_seqs=n_seqs, cols=cols, page=page, n_kv=1, seed=cols)
    r = np.random.default_rng(cols)

    def lengths():
        return [int(v) for v in r.integers(0, cols * page + 1, n_seqs)]

    t.resize(lengths())
    t.resize(lengths())
    new = lengths()
    half = [0 if i % 2 else -1 for i in range(n_seqs)]
    t.resize(half)
    pairs = [(i, i + 1) for i in range(0, n_seqs - 1, 2)]
    t.fork([a for a, _ in pairs], [b for _, b in pairs])
    t.resize(new)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n_seqs,cols", [(3, 8), (80, 1000)])
def test_free_pages_far_up_in_a_large_pool(n_seqs, cols):
    """The first 208000 pages are the caller's own (no holder, not free)."""
    t = Both(n_pages=250000, n_seqs=n_seqs, cols=cols, page=1, n_kv=1)
    t.free[:6500] = 0
    t.m.free = set(range(6500 * 32, 250000))
    t.resize([5] + [0] * (n_seqs - 2) + [cols])
    t.resize([3] + [2] * (n_seqs - 2) + [cols // 2])
    t.fork([0], [0])
    t.resize([cols] * n_seqs)
    assert t.resize([0] * n_seqs) == 0 and len(t.m.free) == 250000 - 6500 * 32


def test_workspaces_of_any_content():
    import torch
    need = B.kv_resize_workspace_bytes(5, 70)
    for fill in (0, 255):
        t = Both()
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        t.resize([17, 0, 16, 1, 144], workspace=ws)
        t.resize([18, 40, 0, 1, 1], workspace=ws)


# ---------------------------------------------------------------------------- copies

def pool(n_pages, n_kv, page, dim, layout, seed, dt):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "heads":
        return [torch.randn(n_pages, n_kv, page, dim, generator=g, device="cuda").to(dt) for _ in range(2)]
    if layout == "tokens":
        return [torch.randn(n_pages, page, n_kv, dim, generator=g, device="cuda").to(dt).transpose(1, 2) for _ in range(2)]
    both = torch.randn(n_pages, n_kv, page, 2 * dim + 8, generator=g, device="cuda").to(dt)
    return [both[..., :dim], both[..., dim: 2 * dim]]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,n_kv", [(1, 1), (16, 8), (7, 3), (300, 2)])
@pytest.mark.parametrize("a,b", [("heads", "heads"), ("tokens", "heads"), ("beside", "tokens")])
def test_copies(dim, page, n_kv, a, b):
    import torch
    src, dst = pool(9, n_kv, page, dim, a, 1, torch.float16), pool(12, n_kv, page, dim, b, 2, torch.float16)
    want = [d.clone() for d in dst]
    f, to = [3, 8, 0, -1, 9, 4, 5, 3], [11, 0, 5, 1, 2, 12, -1, 7]         # the fourth to seventh do not exist
    for i, j in zip(f[:3] + f[7:], to[:3] + to[7:]):
        for s, w in zip(src, want):
            w[j] = s[i]
    kept = [s.clone() for s in src]
    B.q2_0_kv_copy(*dst, *src, torch.tensor(f, dtype=torch.int32, device="cuda"), torch.tensor(to, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(dst + src, want + kept))


def test_copies_within_a_pool():
    import torch
    k, v = pool(6, 2, 16, 64, "heads", 3, torch.bfloat16)
    want = [k.clone(), v.clone()]
    for w in want:
        w[0], w[5] = w[2].clone(), w[2].clone()
    ints = dict(dtype=torch.int32, device="cuda")
    B.q2_0_kv_copy(k, v, k, v, torch.tensor([2, 2], **ints), torch.tensor([0, 5], **ints))
    B.q2_0_kv_copy(k, v, k, v, torch.tensor([], **ints), torch.tensor([], **ints))
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_pages_past_32_bit_offsets():
    import torch
    n = 17000                                # 17000 pages of 128 KiB of keys: 2.2 GB each, elements past 2^30, bytes past 2^31
    k, v = (torch.empty(n, 8, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[[5, n - 1]], v[[5, n - 1]] = 1.5, 2.5
    k[[7, n - 2]], v[[7, n - 2]] = -1.0, -2.0
    ints = dict(dtype=torch.int32, device="cuda")
    B.q2_0_kv_copy(k, v, k, v, torch.tensor([5, n - 1], **ints), torch.tensor([n - 2, 7], **ints))
    torch.cuda.synchronize()
    for p in (5, 7, n - 2, n - 1):
        assert torch.all(k[p] == 1.5) and torch.all(v[p] == 2.5)


# ---------------------------------------------------------------------------- compact

@pytest.mark.parametrize("n_pages,to_pages,layout", [(70, 40, "heads"), (64, 200, "tokens"), (31, 31, "beside"), (1, 1, "heads"),
                                                     (5000, 3001, "heads"), (8192, 700, "tokens"), (8193, 9000, "heads")])
def test_compact(n_pages, to_pages, layout):
    import torch
    r = random.Random(n_pages)
    n_seqs, cols, page, n_kv, dim = 6, 40, 5, 2, 64
    used = sorted(r.sample(range(n_pages), min(n_pages, to_pages) * 3 // 4 or 1))
    ref = [0] * n_pages
    for p in used:
        ref[p] = r.randint(0, 3)             # (0: the caller's own)
    table = [[r.choice(used) for _ in range(cols)] for _ in range(n_seqs)]
    lens = [0, 1, page * cols, 77, -4, page * cols + 1]
    table[3][2], table[3][3], table[2][0] = -1, n_pages, next((p for p in range(n_pages) if p not in used), -1)
    src, dst = pool(n_pages, n_kv, page, dim, layout, 1, torch.bfloat16), pool(to_pages, n_kv, page, dim, "heads", 2, torch.bfloat16)
    ints = dict(dtype=torch.int32, device="cuda")
    free = words(set(range(n_pages)) - set(used), n_pages)
    if n_pages % 32:
        free = free | np.array([0] * (len(free) - 1) + [-(1 << (n_pages % 32))], np.int64).astype(np.int32)   # bits past the pool
    dev = dict(ref=torch.tensor(ref, **ints), free=torch.tensor(free, device="cuda"), table=torch.tensor(table, **ints),
               lens=torch.tensor(lens, **ints))
    ref_to, free_to = B.q2_0_kv_pages(to_pages)
    ref_to.fill_(77)
    wide = torch.full((n_seqs, cols + 3), 55, **ints)
    want = [d.clone() for d in dst]
    for w, s in zip(want, src):
        w[: len(used)] = s[used]
    n_used = B.q2_0_kv_compact(*dst, ref_to, free_to, wide[:, :cols], *src, **dev)
    torch.cuda.synchronize()
    assert n_used.item() == len(used)
    assert all(torch.equal(x, y) for x, y in zip(dst, want))
    assert ref_to.tolist() == [ref[p] for p in used] + [0] * (to_pages - len(used))
    assert np.array_equal(free_to.cpu().numpy(), words(range(len(used), to_pages), to_pages))
    number = {p: i for i, p in enumerate(used)}
    rows = [[number.get(p, -1) if 0 <= n <= cols * page and i * page < n else -1 for i, p in enumerate(row)]
            for row, n in zip(table, lens)]
    assert wide[:, :cols].tolist() == rows and torch.all(wide[:, cols:] == 55)


def test_compact_into_too_small_a_pool():
    import torch
    src, dst = pool(20, 1, 4, 64, "heads", 1, torch.float16), pool(8, 1, 4, 64, "heads", 2, torch.float16)
    ints = dict(dtype=torch.int32, device="cuda")
    ref, free = torch.ones(20, **ints), torch.tensor([0b11], **ints)
    ref_to, free_to = B.q2_0_kv_pages(8)
    table, table_to = torch.full((2, 3), 5, **ints), torch.full((2, 3), -9, **ints)
    want = [d.clone() for d in dst]
    n_used = B.q2_0_kv_compact(*dst, ref_to, free_to, table_to, *src, ref, free, table, torch.tensor([4, 9], **ints))
    torch.cuda.synchronize()
    assert n_used.item() == 18 and all(torch.equal(x, y) for x, y in zip(dst, want))
    assert torch.all(ref_to == 0) and torch.all(free_to == -1) and torch.all(table_to == -9)


def test_compact_of_nothing():
    import torch
    src, dst = pool(40, 1, 4, 64, "heads", 1, torch.float16), pool(3, 1, 4, 64, "heads", 2, torch.float16)
    (ref, free), (ref_to, free_to) = B.q2_0_kv_pages(40), B.q2_0_kv_pages(3)
    none = torch.zeros(0, 5, dtype=torch.int32, device="cuda")
    n_used = B.q2_0_kv_compact(*dst, ref_to, free_to, none.clone(), *src, ref, free, none, none[:, 0])
    torch.cuda.synchronize()
    assert n_used.item() == 0 and free_to.tolist() == [7] and torch.all(ref_to == 0)
