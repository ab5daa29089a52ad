// C ABI of the decoder-step operators: argument validation and dispatch.  As for the
// products, every check runs on the host before anything is launched, in the order SHAPE,
// the empty no-op, NULL, LAYOUT, UNSUPPORTED, ALIGN, WORKSPACE.
#include <cmath>

#include "../../include/q2_0.h"
#include "layer_common.h"

namespace {

constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxStride = (int64_t)1 << 40;     // elements; byte offsets stay far inside 63 bits
constexpr int64_t kMaxQueryRows = (int64_t)1 << 28;
constexpr int64_t kMaxTokenStride = (int64_t)1 << 24;
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads: a launch counts threads in 32 bits

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

bool known_act(int t) { return t == Q2_0_ACT_F32 || t == Q2_0_ACT_F16 || t == Q2_0_ACT_BF16; }

bool cache_shape_ok(const q2_0_kv_cache &c) {
    return in(c.n_pages, 0, kMaxInt) && in(c.page_size, 1, kMaxInt) && in(c.n_kv, 1, 4096) && in(c.head_dim, 1, 4096);
}

int check_cache(const q2_0_kv_cache &c) {
    if (!c.k || !c.v) return Q2_0_ERR_NULL;
    for (const int64_t st : {c.page_stride, c.head_stride, c.token_stride})
        if (!in(st, 8, kMaxStride) || st % 8 != 0) return Q2_0_ERR_LAYOUT;
    if (c.token_stride > kMaxTokenStride || c.token_stride < c.head_dim || c.head_stride < c.head_dim)
        return Q2_0_ERR_LAYOUT;
    return Q2_0_OK;
}

bool cache_known(const q2_0_kv_cache &c) {
    return (c.type == Q2_0_ACT_F16 || c.type == Q2_0_ACT_BF16) &&
           (c.head_dim == 64 || c.head_dim == 128 || c.head_dim == 256);
}

bool table_ok(int64_t n_seqs, int64_t table_len) { return in(n_seqs, 0, kMaxInt) && in(table_len, 0, kMaxInt); }

bool attn_sizes_ok(int64_t n_seqs, int64_t n_q, int64_t n_kv, int64_t n_qt, int64_t prefix_len, int64_t max_len) {
    if (!in(n_seqs, 0, 1 << 20) || !in(n_kv, 1, 4096) || !in(n_q, 0, 4096) || n_q % n_kv != 0) return false;
    if (n_seqs * n_q > kMaxQueryRows / Q2_0_ATTN_MAX_QT) return false;   // 32-bit rows and launch grids
    if (!in(n_qt, 1, Q2_0_ATTN_MAX_QT) || !in(max_len, 0, kMaxInt - 64) || !in(prefix_len, 0, max_len)) return false;
    return true;
}

bool moe_sizes_ok(int64_t n_ff, int64_t K, int64_t n_used, int64_t n_tokens) {
    return in(n_ff, 64, (int64_t)1 << 20) && n_ff % 64 == 0 && in(K, 64, (int64_t)1 << 20) && K % 64 == 0 &&
           in(n_used, 0, kMaxInt) && in(n_tokens, 0, kMaxInt);
}

}  // namespace

extern "C" {

int q2_0_kv_append(const q2_0_kv_cache *cache, const int32_t *table, int64_t n_seqs, int64_t table_len,
                   int64_t ld_table, const int32_t *seq, const int32_t *pos, int64_t n_tokens, const void *q,
                   int64_t ldq, int64_t n_q, const void *k, int64_t ldk, const void *v, int64_t ldv, int x_type,
                   const float *rope, int64_t n_pos, int64_t rot_dim, int style, void *q_out, int64_t ldqo,
                   void *stream) {
    if (!cache) return Q2_0_ERR_NULL;
    const q2_0_kv_cache &c = *cache;
    if (!cache_shape_ok(c) || !table_ok(n_seqs, table_len) || !in(n_q, 0, 4096) || !in(n_tokens, 0, kMaxInt))
        return Q2_0_ERR_SHAPE;
    if (!in(rot_dim, 0, c.head_dim) || rot_dim % 2 != 0 || !in(n_pos, 0, kMaxInt)) return Q2_0_ERR_SHAPE;
    if (n_tokens * ((n_q + 2 * c.n_kv) * c.head_dim / 512 + 1) > kMaxInt) return Q2_0_ERR_SHAPE;   // launch grid
    if (n_tokens == 0) return Q2_0_OK;
    if (!table || !seq || !pos || !k || !v || (rot_dim > 0 && !rope) || (n_q > 0 && (!q || !q_out))) return Q2_0_ERR_NULL;
    int st = check_cache(c);
    if (st) return st;
    if (ld_table < table_len || ldk < c.n_kv * c.head_dim || ldv < c.n_kv * c.head_dim ||
        (n_q > 0 && (ldq < n_q * c.head_dim || ldqo < n_q * c.head_dim)))
        return Q2_0_ERR_LAYOUT;
    if (!known_act(x_type) || !cache_known(c) || (style != Q2_0_ROPE_HALF && style != Q2_0_ROPE_PAIRS))
        return Q2_0_ERR_UNSUPPORTED;
    const uintptr_t eb = q2_0::act_bytes((q2_0::Act)x_type);
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(table, 4) || !aligned(seq, 4) || !aligned(pos, 4) ||
        !aligned(k, eb) || !aligned(v, eb) || (rot_dim > 0 && !aligned(rope, 4)) ||
        (n_q > 0 && (!aligned(q, eb) || !aligned(q_out, 2))))
        return Q2_0_ERR_ALIGN;
    q2_0::KvAppend a;
    a.q = q, a.k = k, a.v = v;
    a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.q_out = q_out, a.ldqo = ldqo;
    a.kc = c.k, a.vc = c.v;
    a.page_stride = c.page_stride, a.head_stride = c.head_stride, a.token_stride = c.token_stride;
    a.table = table, a.ld_table = ld_table, a.n_seqs = n_seqs, a.table_len = table_len, a.n_pages = c.n_pages;
    a.seq = seq, a.pos = pos;
    a.rope = rope, a.n_pos = n_pos;
    a.page = q2_0::FastDiv::make((uint32_t)c.page_size);
    a.n_q = (int)n_q, a.n_kv = (int)c.n_kv, a.dim = (int)c.head_dim, a.rot = (int)rot_dim;
    a.half_style = style == Q2_0_ROPE_HALF;
    a.head_blocks = 0;
    // (a SHAPE error too, but of the variant that alignment decides)
    if (q2_0::kv_append_groups(a, (q2_0::Act)x_type, n_tokens) > kMaxGroups) return Q2_0_ERR_SHAPE;
    return q2_0::record_hip_error(q2_0::launch_kv_append(a, (q2_0::Act)x_type, (q2_0::Act)c.type, n_tokens,
                                                         static_cast<hipStream_t>(stream)));
}

size_t q2_0_attn_shared_workspace_bytes(int64_t n_seqs, int64_t n_q, int64_t n_kv, int64_t head_dim, int64_t n_qt,
                                        int64_t prefix_len, int64_t max_len) {
    if (!attn_sizes_ok(n_seqs, n_q, n_kv, n_qt, prefix_len, max_len) || n_seqs == 0 || n_q == 0) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return q2_0::attn_plan(n_seqs, n_q, n_kv, head_dim, n_qt, prefix_len, max_len).ws_bytes;
}

int q2_0_attn_shared(const q2_0_kv_cache *cache, const int32_t *table, int64_t n_seqs, int64_t table_len,
                     int64_t ld_table, const int32_t *lens, int64_t prefix_len, int64_t max_len, const void *q,
                     int64_t ldq, int64_t n_q, int64_t n_qt, float scale, void *out, int64_t ldo, void *workspace,
                     size_t ws_bytes, void *stream) {
    if (!cache) return Q2_0_ERR_NULL;
    const q2_0_kv_cache &c = *cache;
    if (!cache_shape_ok(c) || !table_ok(n_seqs, table_len) ||
        !attn_sizes_ok(n_seqs, n_q, c.n_kv, n_qt, prefix_len, max_len) || max_len > table_len * c.page_size ||
        (max_len > 0 && c.n_pages == 0) || !std::isfinite(scale) || !(scale > 0.f))
        return Q2_0_ERR_SHAPE;
    if (n_seqs == 0 || n_q == 0) return Q2_0_OK;
    const q2_0::AttnPlan p = q2_0::attn_plan(n_seqs, n_q, c.n_kv, c.head_dim, n_qt, prefix_len, max_len);
    if (p.groups > kMaxGroups) return Q2_0_ERR_SHAPE;
    if (!lens || !q || !out || (max_len > 0 && !table)) return Q2_0_ERR_NULL;
    int st = check_cache(c);
    if (st) return st;
    if (ld_table < table_len || ldq < n_q * c.head_dim || ldo < n_q * c.head_dim || ldq % 8 != 0 || ldo % 8 != 0)
        return Q2_0_ERR_LAYOUT;
    if (!cache_known(c)) return Q2_0_ERR_UNSUPPORTED;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) ||
        !aligned(lens, 4))
        return Q2_0_ERR_ALIGN;
    if (p.ws_bytes && (ws_bytes < p.ws_bytes || !workspace || !aligned(workspace, 16))) return Q2_0_ERR_WORKSPACE;
    q2_0::AttnShared a{};
    a.q = q, a.ldq = ldq;
    a.kc = c.k, a.vc = c.v;
    a.page_stride = c.page_stride, a.head_stride = c.head_stride, a.token_stride = c.token_stride;
    a.table = table, a.ld_table = ld_table, a.n_pages = c.n_pages;
    a.lens = lens;
    a.out = out, a.ldo = ldo;
    a.part_o = static_cast<float *>(workspace);
    a.page = q2_0::FastDiv::make((uint32_t)c.page_size);
    a.group = q2_0::FastDiv::make((uint32_t)(n_q / c.n_kv));
    a.scale2 = scale * 1.44269504088896340736f;
    a.n_seqs = (int)n_seqs, a.n_qt = (int)n_qt, a.n_q = (int)n_q, a.n_kv = (int)c.n_kv;
    a.prefix_len = (int)prefix_len, a.max_len = (int)max_len;
    return q2_0::record_hip_error(q2_0::launch_attn_shared(a, p, (q2_0::Act)c.type, (int)c.head_dim,
                                                           static_cast<hipStream_t>(stream)));
}

int q2_0_moe_route(const void *logits, int x_type, int64_t ld, int64_t n_tokens, int64_t n_expert, int64_t n_used,
                   int normalise, int32_t *ids, float *weights, void *stream) {
    if (!in(n_tokens, 0, 4 * kMaxGroups) || !in(n_expert, 1, 8192) || !in(n_used, 1, 64) || n_used > n_expert)
        return Q2_0_ERR_SHAPE;
    if (n_tokens == 0) return Q2_0_OK;
    if (!logits || !ids || !weights) return Q2_0_ERR_NULL;
    if (ld < n_expert) return Q2_0_ERR_LAYOUT;
    if (!known_act(x_type)) return Q2_0_ERR_UNSUPPORTED;
    if (!aligned(logits, q2_0::act_bytes((q2_0::Act)x_type)) || !aligned(ids, 4) || !aligned(weights, 4))
        return Q2_0_ERR_ALIGN;
    return q2_0::record_hip_error(q2_0::launch_moe_choose(logits, (q2_0::Act)x_type, ld, n_tokens, (int)n_expert,
                                                          (int)n_used, normalise, ids, weights,
                                                          static_cast<hipStream_t>(stream)));
}

size_t q2_0_moe_layer_workspace_bytes(int64_t n_ff, int64_t K, int64_t n_used, int64_t n_tokens) {
    if (!moe_sizes_ok(n_ff, K, n_used, n_tokens) || n_used > Q2_0_MOE_LAYER_MAX_USED ||
        n_tokens > Q2_0_MOE_LAYER_MAX_TOKENS)
        return 0;
    return q2_0::moe_layer_ws_bytes(n_ff, K, n_used, n_tokens);
}

int q2_0_moe_layer(const void *w_gate, const void *w_up, const void *w_down, int64_t n_expert, int64_t n_ff,
                   int64_t K, const void *x, int x_type, int64_t ldx, const int32_t *ids, const float *weights,
                   int64_t n_used, int64_t n_tokens, float *y, int64_t ldy, void *workspace, size_t ws_bytes,
                   void *stream) {
    if (!moe_sizes_ok(n_ff, K, n_used, n_tokens) || !in(n_expert, 1, 8192)) return Q2_0_ERR_SHAPE;
    if (n_tokens == 0) return Q2_0_OK;
    if (!y || (n_used > 0 && (!w_gate || !w_up || !w_down || !x || !ids || !weights))) return Q2_0_ERR_NULL;
    if (ldx < K || ldy < K) return Q2_0_ERR_LAYOUT;
    if (!known_act(x_type) || n_used > Q2_0_MOE_LAYER_MAX_USED || n_tokens > Q2_0_MOE_LAYER_MAX_TOKENS)
        return Q2_0_ERR_UNSUPPORTED;
    if (!aligned(w_gate, 2) || !aligned(w_up, 2) || !aligned(w_down, 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(x, q2_0::act_bytes((q2_0::Act)x_type)) || !aligned(y, 4))
        return Q2_0_ERR_ALIGN;
    const size_t need = q2_0_moe_layer_workspace_bytes(n_ff, K, n_used, n_tokens);
    if (need && (ws_bytes < need || !workspace || !aligned(workspace, 16))) return Q2_0_ERR_WORKSPACE;
    return q2_0::record_hip_error(q2_0::launch_moe_layer(
        static_cast<const uint8_t *>(w_gate), static_cast<const uint8_t *>(w_up), static_cast<const uint8_t *>(w_down),
        (int)n_expert, (int)n_ff, (int)K, x, (q2_0::Act)x_type, ldx, ids, weights, (int)n_used, (int)n_tokens, y, ldy,
        workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
