"""Argument checks of the operators between two decoder steps on the host: every call here fails validation or is
an empty no-op, so nothing is launched and no GPU is needed."""

import os
import subprocess
import sys

import pytest
from test_abi_layer import BF16, F16, F32, P, cache

from ternary_bit_quantized_amd import build as BUILD
from ternary_bit_quantized_amd import q2_0 as B

Q = P + (1 << 30)      # another fake address
BIG = 1 << 40


def route(**kw):
    a = dict(logits=P, x_type=F32, ld=128, n_tokens=3, n_expert=128, n_used=8, score=1, bias=P, n_group=8, n_group_used=4,
             group_top=2, normalise=1, scale=2.5, ids=P, weights=P)
    a.update(kw)
    return B.moe_route_groups_raw(**a)


def test_route_groups():
    assert route(n_expert=0) == route(n_expert=1025, ld=2000, n_group=1, n_group_used=1) == B.Q2_0_ERR_SHAPE
    assert route(n_used=0) == route(n_used=65) == B.Q2_0_ERR_SHAPE
    assert route(n_used=17, n_group_used=1) == B.Q2_0_ERR_SHAPE           # more than the open groups hold
    assert route(n_used=16, n_group_used=1, logits=0) == B.Q2_0_ERR_NULL
    assert route(n_group=0) == route(n_group=65) == route(n_group=7) == B.Q2_0_ERR_SHAPE
    assert route(n_group_used=0) == route(n_group_used=9) == B.Q2_0_ERR_SHAPE
    assert route(group_top=0) == route(group_top=3) == B.Q2_0_ERR_SHAPE
    assert route(n_expert=8, n_used=2, group_top=2) == B.Q2_0_ERR_SHAPE   # groups of one expert
    assert route(scale=float("nan")) == route(scale=float("inf")) == B.Q2_0_ERR_SHAPE
    assert route(n_tokens=-1) == route(n_tokens=(1 << 26) - 3) == B.Q2_0_ERR_SHAPE
    assert route(n_tokens=(1 << 26) - 4, logits=0) == B.Q2_0_ERR_NULL
    assert route(n_tokens=0, logits=0, ids=0, weights=0) == B.Q2_0_OK
    for name in ("logits", "ids", "weights"):
        assert route(**{name: 0}) == B.Q2_0_ERR_NULL, name
    assert route(ld=127) == B.Q2_0_ERR_LAYOUT
    assert route(x_type=3) == route(score=2) == B.Q2_0_ERR_UNSUPPORTED
    for name in ("logits", "bias", "ids", "weights"):
        assert route(**{name: P + 2}) == B.Q2_0_ERR_ALIGN, name
    assert route(x_type=F16, logits=P + 1) == B.Q2_0_ERR_ALIGN


def verify(**kw):
    a = dict(target=P, ld_target=1000, draft=P, ld_draft=1000, x_type=F32, form=0, n_vocab=1000, temperature=P, tokens=P, n_draft=P,
             u=P, n_seqs=3, max_draft=4, out=P, n_accepted=P, workspace=P, ws_bytes=BIG)
    a.update(kw)
    return B.draft_verify_raw(**a)


def test_draft_verify():
    assert verify(n_seqs=-1) == verify(n_seqs=(1 << 20) + 1) == B.Q2_0_ERR_SHAPE
    assert verify(max_draft=-1) == verify(max_draft=B.DRAFT_MAX + 1) == B.Q2_0_ERR_SHAPE
    assert verify(n_vocab=0) == verify(n_vocab=(1 << 24) + 1, ld_target=BIG, ld_draft=BIG) == B.Q2_0_ERR_SHAPE
    # launches past 2^24 workgroups: 2^20 sequences of 9 rows of 2 chunks
    assert verify(n_seqs=1 << 20, n_vocab=40000, ld_target=40000, ld_draft=40000) == B.Q2_0_ERR_SHAPE
    assert verify(n_seqs=0, target=0, out=0, n_accepted=0, u=0, n_draft=0, tokens=0) == B.Q2_0_OK
    for name in ("target", "n_draft", "u", "out", "n_accepted", "tokens"):
        assert verify(**{name: 0}) == B.Q2_0_ERR_NULL, name
    assert verify(tokens=0, max_draft=0, ws_bytes=0) == B.Q2_0_ERR_WORKSPACE   # nothing drafted: no tokens
    assert verify(draft=0, ws_bytes=0) == verify(temperature=0, ws_bytes=0) == B.Q2_0_ERR_WORKSPACE
    assert verify(ld_target=999) == verify(ld_draft=999) == B.Q2_0_ERR_LAYOUT
    assert verify(ld_draft=0, draft=0, ws_bytes=0) == B.Q2_0_ERR_WORKSPACE
    assert verify(x_type=4) == verify(form=2) == verify(form=1) == B.Q2_0_ERR_UNSUPPORTED   # (probabilities have no temperature)
    for name in ("target", "draft", "temperature", "tokens", "n_draft", "u", "out", "n_accepted"):
        assert verify(**{name: P + 2}) == B.Q2_0_ERR_ALIGN, name
    assert verify(x_type=BF16, target=P + 1) == B.Q2_0_ERR_ALIGN
    for form, xt, has in ((0, F32, 1), (0, F16, 0), (1, F32, 1)):
        need = B.draft_verify_workspace_bytes(3, 4, 1000, xt, form, has)
        assert need > 0
        kw = dict(x_type=xt, form=form, draft=P if has else 0, temperature=0)
        assert verify(ws_bytes=need - 1, **kw) == verify(workspace=0, **kw) == verify(workspace=P + 8, **kw) == B.Q2_0_ERR_WORKSPACE
    assert B.draft_verify_workspace_bytes(0, 4, 1000, F32, 0, 1) == B.draft_verify_workspace_bytes(3, 16, 1000, F32, 0, 1) == 0
    assert B.draft_verify_workspace_bytes(3, 4, 1000, 5, 0, 1) == B.draft_verify_workspace_bytes(3, 4, 1000, F32, 3, 1) == 0


def copy(to=None, frm=None, src=P, dst=P, n=5):
    return B.kv_copy_raw(cache() if to is None else to, cache(k=Q, v=Q) if frm is None else frm, src, dst, n)


def pages(ref=P, free=P, n_pages=10):
    return B.KvPages(ref, free, n_pages)


def resize(c=None, p=None, **kw):
    a = dict(table=P, n_seqs=3, table_len=4, ld_table=4, lens=P, new_lens=P, missing=P, workspace=P, ws_bytes=BIG)
    a.update(kw)
    return B.kv_resize_raw(cache() if c is None else c, pages() if p is None else p, **a)


def fork(**kw):
    a = dict(ref=P, n_pages=10, table=P, n_seqs=3, table_len=4, ld_table=4, page_size=16, lens=P, src=P, dst=P, n=2, workspace=P,
             ws_bytes=BIG)
    a.update(kw)
    return B.kv_fork_raw(**a)


def compact(to=None, tp=None, frm=None, fp=None, **kw):
    a = dict(table=P, n_seqs=3, table_len=4, ld_table=4, lens=P, to_table=Q, ld_to_table=4, n_used=P, workspace=P, ws_bytes=BIG)
    a.update(kw)
    return B.kv_compact_raw(cache(k=Q, v=Q + 64) if to is None else to, pages(Q, Q) if tp is None else tp,
                            cache(k=P, v=P + 64) if frm is None else frm, pages() if fp is None else fp, **a)


@pytest.mark.parametrize("call", [lambda c: copy(to=c), lambda c: copy(frm=c), lambda c: resize(c), lambda c: compact(to=c),
                                  lambda c: compact(frm=c)])
def test_cache_checks(call):
    assert call(cache(page_size=0)) == call(cache(n_kv=0)) == call(cache(n_pages=-1)) == B.Q2_0_ERR_SHAPE
    assert call(cache(n_pages=(1 << 30) + 1)) == B.Q2_0_ERR_SHAPE
    assert call(cache(page_size=(1 << 31) // 64)) == B.Q2_0_ERR_SHAPE     # 2^31 vectors a page
    assert call(cache(k=0)) == call(cache(v=0)) == B.Q2_0_ERR_NULL
    for kw in (dict(token_stride=127), dict(token_stride=64), dict(token_stride=(1 << 24) + 8), dict(page_stride=0),
               dict(head_stride=(1 << 40) + 8), dict(head_stride=64)):
        assert call(cache(k=Q + 32, v=Q + 96, **kw)) == B.Q2_0_ERR_LAYOUT, kw
    assert call(cache(type=9, k=Q + 32, v=Q + 96)) == B.Q2_0_ERR_UNSUPPORTED
    assert call(cache(k=Q + 8, v=Q + 72)) == B.Q2_0_ERR_ALIGN


def test_copy():
    assert B.kv_copy_raw(None, cache(), P, P, 1) == B.kv_copy_raw(cache(), None, P, P, 1) == B.Q2_0_ERR_NULL
    for kw in (dict(page_size=8), dict(n_kv=4), dict(head_dim=64)):
        assert copy(frm=cache(**kw)) == B.Q2_0_ERR_SHAPE                  # other pages
    assert copy(n=-1) == copy(n=1 << 24) == B.Q2_0_ERR_SHAPE
    assert copy(n=(1 << 24) - 1, src=0) == B.Q2_0_ERR_NULL                # one workgroup a page of these
    assert copy(n=0, src=0, dst=0) == B.Q2_0_OK
    assert copy(src=0) == copy(dst=0) == B.Q2_0_ERR_NULL
    assert copy(frm=cache(type=F16)) == B.Q2_0_ERR_UNSUPPORTED            # types differ
    odd = dict(head_dim=96, token_stride=128)
    assert copy(to=cache(**odd), frm=cache(**odd)) == B.Q2_0_ERR_UNSUPPORTED
    assert copy(src=P + 2) == copy(dst=P + 2) == B.Q2_0_ERR_ALIGN


def test_resize():
    assert B.kv_resize_raw(None, pages(), P, 1, 1, 1, P, P, P, P, BIG) == B.Q2_0_ERR_NULL
    assert B.kv_resize_raw(cache(), None, P, 1, 1, 1, P, P, P, P, BIG) == B.Q2_0_ERR_NULL
    assert resize(p=pages(n_pages=11)) == B.Q2_0_ERR_SHAPE
    assert resize(n_seqs=-1) == resize(n_seqs=8193) == B.Q2_0_ERR_SHAPE
    assert resize(table_len=-1) == resize(table_len=(1 << 30) + 1) == B.Q2_0_ERR_SHAPE
    assert resize(n_seqs=8192, table_len=1 << 21, ld_table=1 << 21) == B.Q2_0_ERR_SHAPE      # launch grid
    assert resize(n_seqs=0, table=0, lens=0, new_lens=0, missing=0, ws_bytes=0) == B.Q2_0_OK
    for name in ("table", "lens", "new_lens", "missing"):
        assert resize(**{name: 0}) == B.Q2_0_ERR_NULL, name
    assert resize(p=pages(ref=0)) == resize(p=pages(free=0)) == B.Q2_0_ERR_NULL
    assert resize(ld_table=3) == B.Q2_0_ERR_LAYOUT
    for name in ("table", "lens", "new_lens", "missing"):
        assert resize(**{name: P + 2}) == B.Q2_0_ERR_ALIGN, name
    assert resize(p=pages(ref=P + 2)) == resize(p=pages(free=P + 1)) == B.Q2_0_ERR_ALIGN
    need = B.kv_resize_workspace_bytes(3, 10)
    assert need > 0
    assert resize(ws_bytes=need - 1) == resize(workspace=0) == resize(workspace=P + 8) == B.Q2_0_ERR_WORKSPACE
    assert B.kv_resize_workspace_bytes(8193, 10) == B.kv_resize_workspace_bytes(3, -1) == 0


def test_fork():
    assert fork(n_seqs=-1) == fork(table_len=-1) == fork(n_pages=-1) == fork(page_size=0) == fork(n=-1) == B.Q2_0_ERR_SHAPE
    assert fork(n=1 << 24) == fork(n_pages=(1 << 30) + 1) == B.Q2_0_ERR_SHAPE
    assert fork(n=(1 << 24) - 1, ref=0) == B.Q2_0_ERR_NULL
    assert fork(n=0, ref=0, table=0, lens=0, src=0, dst=0, ws_bytes=0) == fork(n_seqs=0, src=0, ws_bytes=0) == B.Q2_0_OK
    for name in ("ref", "table", "lens", "src", "dst"):
        assert fork(**{name: 0}) == B.Q2_0_ERR_NULL, name
        assert fork(**{name: P + 2}) == B.Q2_0_ERR_ALIGN, name
    assert fork(ld_table=3) == B.Q2_0_ERR_LAYOUT
    need = B.kv_fork_workspace_bytes(2)
    assert need > 0
    assert fork(ws_bytes=need - 1) == fork(workspace=0) == fork(workspace=P + 4) == B.Q2_0_ERR_WORKSPACE


def test_compact():
    L = B.lib()
    for i in range(4):
        assert L.q2_0_kv_compact(*([None] * 5), 0, 0, 0, *([None] * 2), 0, P, P, BIG, None) == B.Q2_0_ERR_NULL
    for kw in (dict(page_size=8), dict(n_kv=4), dict(head_dim=64)):
        assert compact(frm=cache(k=P, v=P + 64, **kw)) == B.Q2_0_ERR_SHAPE
    assert compact(tp=pages(Q, Q, 9)) == compact(fp=pages(n_pages=11)) == compact(n_seqs=-1) == B.Q2_0_ERR_SHAPE
    many = (1 << 24) - 3
    assert compact(frm=cache(n_pages=many, k=P, v=P + 64), fp=pages(n_pages=many)) == B.Q2_0_ERR_SHAPE
    for name in ("table", "lens", "to_table", "n_used"):
        assert compact(**{name: 0}) == B.Q2_0_ERR_NULL, name
        assert compact(**{name: Q + 6}) == B.Q2_0_ERR_ALIGN, name
    for bad in (pages(ref=0), pages(free=0)):
        assert compact(fp=bad) == compact(tp=bad) == B.Q2_0_ERR_NULL
    assert compact(fp=pages(P + 2)) == compact(tp=pages(Q, Q + 1)) == B.Q2_0_ERR_ALIGN
    assert compact(ld_table=3) == compact(ld_to_table=3) == B.Q2_0_ERR_LAYOUT
    # nothing of the one pool may be the other's
    assert compact(to=cache(k=P, v=Q)) == compact(to=cache(k=Q, v=P + 64)) == compact(to=cache(k=P + 64, v=Q)) == B.Q2_0_ERR_LAYOUT
    assert compact(tp=pages(P, Q)) == compact(tp=pages(Q, P)) == compact(to_table=P) == B.Q2_0_ERR_LAYOUT
    assert compact(frm=cache(type=F16, k=P, v=P + 64)) == B.Q2_0_ERR_UNSUPPORTED
    need = B.kv_compact_workspace_bytes(10)
    assert need > 0
    assert compact(ws_bytes=need - 1) == compact(workspace=0) == compact(workspace=P + 8) == B.Q2_0_ERR_WORKSPACE
    assert B.kv_compact_workspace_bytes(0) == B.kv_compact_workspace_bytes(-1) == 0

@pytest.mark.parametrize("call", [lambda c: copy(to=c, frm=c, n=1, src=0), lambda c: resize(c, pages(n_pages=1), table=0),
                                  lambda c: compact(to=c, tp=pages(Q, Q, 1), frm=c, fp=pages(n_pages=1), table=0)])
def test_pages_of_nearly_2_31_vectors(call):
    """A thread's last vectors lie up to 2047 past a page's: all of them have to be 32-bit numbers."""
    for kw, vectors in ((dict(n_kv=1, head_dim=64), 16), (dict(n_kv=8, head_dim=128), 256), (dict(n_kv=3, head_dim=256), 192)):
        most = (2 ** 31 - 2048) // vectors
        assert call(cache(n_pages=1, page_size=most + 1, token_stride=256, **kw)) == B.Q2_0_ERR_SHAPE, kw
        assert call(cache(n_pages=1, page_size=(2 ** 31 - 1) // vectors, token_stride=256, **kw)) == B.Q2_0_ERR_SHAPE, kw
    assert copy(to=cache(n_pages=1, page_size=most, token_stride=256, **kw), frm=cache(n_pages=1, page_size=most, token_stride=256, **kw),
                n=1, src=0) == B.Q2_0_ERR_NULL


def test_under_asan_and_ubsan():
    """These tests once more on a build whose host code carries the sanitizers."""
    if os.environ.get("Q2_0_LIB"):
        return
    lib, srcs = os.path.join(BUILD.SAN_DIR, "libq2_0.so"), [os.path.join(BUILD.CSRC, f) for f in os.listdir(BUILD.CSRC)]
    if not os.path.exists(lib) or os.path.getmtime(lib) < max(os.path.getmtime(f) for f in srcs):
        BUILD.build_sanitized()
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       env=BUILD.sanitized_env(), capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    assert r.returncode == 0, text[-4000:]
    assert "ERROR: AddressSanitizer" not in text and "runtime error:" not in text, text[-4000:]
