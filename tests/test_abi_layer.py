"""Argument checks of the decoder-step operators on the host: every call here fails validation
or is an empty no-op, so nothing is launched and no GPU is needed."""

import ctypes

import pytest

from ternary_bit_quantized_amd import q2_0 as B

P = 1 << 20     # a fake, aligned device address: validation never dereferences it
F16, BF16, F32 = B.Q2_0_ACT_F16, B.Q2_0_ACT_BF16, B.Q2_0_ACT_F32


def cache(**kw):
    a = dict(k=P, v=P, type=BF16, n_pages=10, page_size=16, n_kv=2, head_dim=128, page_stride=2 * 16 * 128,
             head_stride=16 * 128, token_stride=128)
    a.update(kw)
    return B.KvCache(*[a[n] for n, _ in B.KvCache._fields_])


def append(c=None, **kw):
    a = dict(table=P, n_seqs=3, table_len=4, ld_table=4, seq=P, pos=P, n_tokens=5, q=P, ldq=512, n_q=4, k=P, ldk=256,
             v=P, ldv=256, x_type=F32, rope=P, n_pos=64, rot_dim=64, style=0, q_out=P, ldqo=512)
    a.update(kw)
    return B.kv_append_raw(cache() if c is None else c, **a)


def attn(c=None, **kw):
    a = dict(table=P, n_seqs=3, table_len=4, ld_table=4, lens=P, prefix_len=0, max_len=64, q=P, ldq=512, n_q=4, n_qt=1,
             scale=0.1, out=P, ldo=512, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return B.attn_shared_raw(cache() if c is None else c, **a)


@pytest.mark.parametrize("call", [append, attn])
def test_cache_checks(call):
    assert call(cache(page_size=0)) == B.Q2_0_ERR_SHAPE
    assert call(cache(n_kv=0)) == B.Q2_0_ERR_SHAPE
    assert call(cache(n_pages=-1)) == B.Q2_0_ERR_SHAPE
    assert call(cache(k=0)) == B.Q2_0_ERR_NULL
    assert call(cache(v=0)) == B.Q2_0_ERR_NULL
    assert call(cache(token_stride=127)) == B.Q2_0_ERR_LAYOUT
    assert call(cache(token_stride=64)) == B.Q2_0_ERR_LAYOUT          # rows would overlap
    assert call(cache(token_stride=(1 << 24) + 8)) == B.Q2_0_ERR_LAYOUT
    assert call(cache(page_stride=0)) == B.Q2_0_ERR_LAYOUT
    assert call(cache(head_stride=(1 << 40) + 8)) == B.Q2_0_ERR_LAYOUT
    assert call(cache(type=F32)) == B.Q2_0_ERR_UNSUPPORTED
    assert call(cache(type=9)) == B.Q2_0_ERR_UNSUPPORTED
    assert call(cache(head_dim=96)) == B.Q2_0_ERR_UNSUPPORTED
    assert call(cache(k=P + 8)) == B.Q2_0_ERR_ALIGN
    assert call(table=P + 2) == B.Q2_0_ERR_ALIGN
    assert call(ld_table=3) == B.Q2_0_ERR_LAYOUT
    assert call(table_len=-1) == B.Q2_0_ERR_SHAPE


def test_null_cache():
    L = B.lib()
    args = [0] * 22
    assert L.q2_0_kv_append(None, *args) == B.Q2_0_ERR_NULL
    assert L.q2_0_attn_shared(None, *([0] * 11), ctypes.c_float(1.0), 0, 0, 0, 0, 0) == B.Q2_0_ERR_NULL


def test_append_checks():
    assert append(n_tokens=-1) == B.Q2_0_ERR_SHAPE
    assert append(rot_dim=7) == B.Q2_0_ERR_SHAPE
    assert append(rot_dim=130) == B.Q2_0_ERR_SHAPE
    assert append(n_pos=-1) == B.Q2_0_ERR_SHAPE
    assert append(n_tokens=(1 << 31) - 1) == B.Q2_0_ERR_SHAPE        # launch grid
    assert append(n_tokens=0, k=0, v=0, q=0, seq=0, pos=0, table=0) == B.Q2_0_OK
    for name in ("table", "seq", "pos", "q", "k", "v", "rope", "q_out"):
        assert append(**{name: 0}) == B.Q2_0_ERR_NULL, name
    assert append(ldk=255) == B.Q2_0_ERR_LAYOUT
    assert append(ldv=255) == B.Q2_0_ERR_LAYOUT
    assert append(ldq=511) == B.Q2_0_ERR_LAYOUT
    assert append(ldqo=511) == B.Q2_0_ERR_LAYOUT
    assert append(x_type=3, k=P + 1) == B.Q2_0_ERR_UNSUPPORTED
    assert append(style=2) == B.Q2_0_ERR_UNSUPPORTED
    assert append(k=P + 2) == B.Q2_0_ERR_ALIGN                        # f32 needs 4 bytes
    assert append(x_type=F16, v=P + 1) == B.Q2_0_ERR_ALIGN
    assert append(rope=P + 2) == B.Q2_0_ERR_ALIGN
    assert append(q_out=P + 1) == B.Q2_0_ERR_ALIGN


def test_attn_checks():
    assert attn(n_q=5) == B.Q2_0_ERR_SHAPE                            # not a multiple of n_kv
    assert attn(n_qt=0) == B.Q2_0_ERR_SHAPE
    assert attn(n_qt=17) == B.Q2_0_ERR_SHAPE
    assert attn(prefix_len=65) == B.Q2_0_ERR_SHAPE
    assert attn(prefix_len=-1) == B.Q2_0_ERR_SHAPE
    assert attn(max_len=65) == B.Q2_0_ERR_SHAPE                       # more than the table holds
    assert attn(cache(n_pages=0)) == B.Q2_0_ERR_SHAPE
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(scale=bad) == B.Q2_0_ERR_SHAPE
    assert attn(n_seqs=0, q=0, out=0, lens=0, table=0) == B.Q2_0_OK
    assert attn(n_q=0, q=0, out=0, lens=0) == B.Q2_0_OK
    for name in ("table", "lens", "q", "out"):
        assert attn(**{name: 0}) == B.Q2_0_ERR_NULL, name
    assert attn(ldq=511) == B.Q2_0_ERR_LAYOUT
    assert attn(ldq=516) == B.Q2_0_ERR_LAYOUT                         # not a multiple of 8
    assert attn(ldo=511) == B.Q2_0_ERR_LAYOUT
    assert attn(q=P + 8) == B.Q2_0_ERR_ALIGN
    assert attn(out=P + 8) == B.Q2_0_ERR_ALIGN
    assert attn(lens=P + 2) == B.Q2_0_ERR_ALIGN
    need = B.attn_shared_workspace_bytes(3, 4, 2, 128, 1, 1000, 2000)
    assert need > 0
    big = dict(table_len=200, ld_table=200, prefix_len=1000, max_len=2000)
    assert attn(ws_bytes=need - 1, **big) == B.Q2_0_ERR_WORKSPACE
    assert attn(workspace=0, **big) == B.Q2_0_ERR_WORKSPACE
    assert attn(workspace=P + 8, **big) == B.Q2_0_ERR_WORKSPACE
    assert B.attn_shared_workspace_bytes(3, 5, 2, 128, 1, 0, 10) == 0
    assert B.attn_shared_workspace_bytes(3, 4, 2, 100, 1, 0, 10) == 0


def test_route_checks():
    def call(logits=P, xt=F32, ld=128, nt=3, ne=128, nu=8, norm=1, ids=P, w=P):
        return B.moe_route_raw(logits, xt, ld, nt, ne, nu, norm, ids, w)

    assert call(ne=0) == B.Q2_0_ERR_SHAPE
    assert call(ne=8193, ld=9000) == B.Q2_0_ERR_SHAPE
    assert call(nu=0) == B.Q2_0_ERR_SHAPE
    assert call(nu=65) == B.Q2_0_ERR_SHAPE
    assert call(ne=4, nu=5) == B.Q2_0_ERR_SHAPE
    assert call(nt=-1) == B.Q2_0_ERR_SHAPE
    assert call(nt=0, logits=0, ids=0, w=0) == B.Q2_0_OK
    assert call(logits=0) == call(ids=0) == call(w=0) == B.Q2_0_ERR_NULL
    assert call(ld=127) == B.Q2_0_ERR_LAYOUT
    assert call(xt=4) == B.Q2_0_ERR_UNSUPPORTED
    assert call(logits=P + 2) == call(ids=P + 2) == call(w=P + 2) == B.Q2_0_ERR_ALIGN


def test_moe_layer_checks():
    def call(wg=P, wu=P, wd=P, ne=4, ff=128, K=192, x=P, xt=F32, ldx=192, ids=P, w=P, nu=2, nt=3, y=P, ldy=192, ws=P,
             wsb=1 << 30):
        return B.moe_layer_raw(wg, wu, wd, ne, ff, K, x, xt, ldx, ids, w, nu, nt, y, ldy, ws, wsb)

    assert call(ff=100) == call(K=100) == call(ff=0) == call(K=0) == B.Q2_0_ERR_SHAPE
    assert call(ne=0) == call(ne=8193) == call(nt=-1) == call(nu=-1) == B.Q2_0_ERR_SHAPE
    assert call(nt=0, x=0, y=0, ids=0, w=0, wg=0) == B.Q2_0_OK
    for name in ("wg", "wu", "wd", "x", "ids", "w", "y"):
        assert call(**{name: 0}) == B.Q2_0_ERR_NULL, name
    assert call(ldx=191) == call(ldy=191) == B.Q2_0_ERR_LAYOUT
    assert call(nt=65) == call(nu=33) == call(xt=7) == B.Q2_0_ERR_UNSUPPORTED
    assert call(wg=P + 1) == call(wu=P + 1) == call(wd=P + 1) == B.Q2_0_ERR_ALIGN
    assert call(x=P + 2) == call(ids=P + 2) == call(w=P + 2) == call(y=P + 2) == B.Q2_0_ERR_ALIGN
    need = B.moe_layer_workspace_bytes(128, 192, 2, 3)
    assert need > 0
    assert call(wsb=need - 1) == call(ws=0) == call(ws=P + 8) == B.Q2_0_ERR_WORKSPACE
    assert B.moe_layer_workspace_bytes(100, 192, 2, 3) == 0
    assert B.moe_layer_workspace_bytes(128, 192, 33, 3) == 0
