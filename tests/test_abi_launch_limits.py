"""Sizes whose launch would have 2^32 threads or more are refused with the other sizes, before anything is
launched: the runtime refuses such a launch only when its turn comes, which for the attention is after its first
kernel.  Every call here fails validation, so no GPU is needed."""

from test_abi_layer import F16, P, append, attn, cache

from ternary_bit_quantized_amd import q2_0 as B


def test_attention():
    # 2^24 query rows of 16 heads; their 2^28 results need joining
    wide = dict(n_seqs=1 << 20, n_qt=16, n_q=16, table_len=300, ld_table=300, prefix_len=3000, max_len=4000, ldq=2048, ldo=2048)
    assert attn(cache(n_pages=1000), **wide) == B.Q2_0_ERR_SHAPE
    assert attn(cache(n_pages=1000), **dict(wide, q=0, workspace=0)) == B.Q2_0_ERR_SHAPE
    assert attn(cache(n_pages=1000), **dict(wide, n_seqs=(1 << 16) - 1, q=0)) == B.Q2_0_ERR_NULL
    # in one part and one split there is nothing to join; 2^20 sequences x 16 heads are 2^24 workgroups
    assert attn(cache(n_pages=1000, n_kv=16), n_seqs=1 << 20, n_q=16, ldq=2048, ldo=2048) == B.Q2_0_ERR_SHAPE
    assert attn(cache(n_pages=1000, n_kv=8), n_seqs=1 << 20, n_q=16, ldq=2048, ldo=2048, q=0) == B.Q2_0_ERR_NULL


def test_append():
    # 8 heads of 128: one workgroup a token, two where rows are aligned to one element only
    assert append(n_tokens=1 << 24) == B.Q2_0_ERR_SHAPE
    assert append(n_tokens=1 << 23, k=P + 4) == B.Q2_0_ERR_SHAPE
    assert append(n_tokens=1 << 23, x_type=F16, ldk=258 + 1) == B.Q2_0_ERR_SHAPE
    assert append(n_tokens=(1 << 24) - 1, k=0) == B.Q2_0_ERR_NULL


def test_route():
    def call(n_tokens, logits=P):
        return B.moe_route_raw(logits, B.Q2_0_ACT_F32, 8, n_tokens, 8, 2, 1, P, P)

    assert call((1 << 26) - 3) == B.Q2_0_ERR_SHAPE
    assert call((1 << 26) - 4, logits=0) == B.Q2_0_ERR_NULL
