// C ABI of the operators between two decoder steps: argument validation and dispatch.  As for the
// others, every check runs on the host before anything is launched, in the order SHAPE, the
// empty no-op, NULL, LAYOUT, UNSUPPORTED, ALIGN, WORKSPACE.
#include <cmath>

#include "../../include/q2_0.h"
#include "serve_common.h"

namespace {

constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxPages = (int64_t)1 << 30;      // and columns of a table: 32-bit places
constexpr int64_t kMaxStride = (int64_t)1 << 40;     // elements; byte offsets stay far inside 63 bits
constexpr int64_t kMaxTokenStride = (int64_t)1 << 24;
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads: a launch counts threads in 32 bits

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

bool known_act(int t) { return t == Q2_0_ACT_F32 || t == Q2_0_ACT_F16 || t == Q2_0_ACT_BF16; }

// 16-byte vectors of a page's keys and values: 2 * n_kv * page_size * head_dim / 8.  A copy's threads count up to the next
// multiple of 2048 of them in 32 bits.
constexpr int64_t kMaxVecs = kMaxInt - 2047;

bool cache_shape_ok(const q2_0_kv_cache &c) {
    return in(c.n_pages, 0, kMaxPages) && in(c.page_size, 1, kMaxInt) && in(c.n_kv, 1, 4096) && in(c.head_dim, 1, 4096) &&
           c.page_size <= kMaxVecs / (c.n_kv * ((c.head_dim + 7) / 8) * 2);
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

bool cache_aligned(const q2_0_kv_cache &c) { return aligned(c.k, 16) && aligned(c.v, 16); }

bool same_pages(const q2_0_kv_cache &a, const q2_0_kv_cache &b) {
    return a.page_size == b.page_size && a.n_kv == b.n_kv && a.head_dim == b.head_dim;
}

bool table_ok(int64_t n_seqs, int64_t table_len) { return in(n_seqs, 0, kMaxInt) && in(table_len, 0, kMaxPages); }

q2_0::PageRows rows_of(const q2_0_kv_cache &c) {
    return q2_0::PageRows{static_cast<char *>(c.k), static_cast<char *>(c.v), c.page_stride * 2, c.head_stride * 2,
                          c.token_stride * 2};
}

q2_0::PageShape shape_of(const q2_0_kv_cache &c) {
    q2_0::PageShape p;
    p.page = q2_0::FastDiv::make((uint32_t)c.page_size);
    p.heads = (int)c.n_kv;
    p.vec_shift = c.head_dim == 64 ? 3 : c.head_dim == 128 ? 4 : 5;
    p.vecs = (int)(2 * c.n_kv * c.page_size * (c.head_dim / 8));
    return p;
}

int64_t copy_groups(const q2_0_kv_cache &c, int64_t n) {
    return c.head_dim % 8 ? 0 : n * ((2 * c.n_kv * c.page_size * (c.head_dim / 8) + 2047) / 2048);
}

int64_t row_groups(int64_t n, int64_t cols) { return n * ((cols + 1023) / 1024); }

q2_0::PageTable table_of(const int32_t *table, int64_t ld, int64_t n_seqs, int64_t cols, const int32_t *lens) {
    return q2_0::PageTable{const_cast<int32_t *>(table), ld, (int)n_seqs, (int)cols, const_cast<int32_t *>(lens)};
}

bool draft_sizes_ok(int64_t n_seqs, int64_t max_draft, int64_t n_vocab) {
    return in(n_seqs, 0, 1 << 20) && in(max_draft, 0, Q2_0_DRAFT_MAX) && in(n_vocab, 1, 1 << 24);
}

}  // namespace

extern "C" {

int q2_0_moe_route_groups(const void *logits, int x_type, int64_t ld, int64_t n_tokens, int64_t n_expert, int64_t n_used,
                          int score, const float *bias, int64_t n_group, int64_t n_group_used, int64_t group_top,
                          int normalise, float scale, int32_t *ids, float *weights, void *stream) {
    if (!in(n_tokens, 0, 4 * kMaxGroups) || !in(n_expert, 1, 1024) || !in(n_used, 1, 64) || !in(n_group, 1, 64) ||
        n_expert % n_group != 0 || !in(n_group_used, 1, n_group) || n_used > n_group_used * (n_expert / n_group) ||
        !in(group_top, 1, 2) || group_top > n_expert / n_group || !std::isfinite(scale))
        return Q2_0_ERR_SHAPE;
    if (n_tokens == 0) return Q2_0_OK;
    if (!logits || !ids || !weights) return Q2_0_ERR_NULL;
    if (ld < n_expert) return Q2_0_ERR_LAYOUT;
    if (!known_act(x_type) || (score != Q2_0_SCORE_SOFTMAX && score != Q2_0_SCORE_SIGMOID)) return Q2_0_ERR_UNSUPPORTED;
    if (!aligned(logits, q2_0::act_bytes((q2_0::Act)x_type)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return Q2_0_ERR_ALIGN;
    q2_0::ChooseGroups a;
    a.logits = logits, a.ld = ld, a.n_tokens = n_tokens;
    a.bias = bias;
    a.size = q2_0::FastDiv::make((uint32_t)(n_expert / n_group));
    a.n_expert = (int)n_expert, a.n_used = (int)n_used;
    a.n_group = (int)n_group, a.n_group_used = (int)n_group_used, a.group_top = (int)group_top;
    a.normalise = normalise, a.scale = scale;
    a.ids = ids, a.weights = weights;
    return q2_0::record_hip_error(q2_0::launch_moe_choose_groups(a, (q2_0::Act)x_type, score == Q2_0_SCORE_SIGMOID,
                                                                 static_cast<hipStream_t>(stream)));
}

size_t q2_0_draft_verify_workspace_bytes(int64_t n_seqs, int64_t max_draft, int64_t n_vocab, int x_type, int form,
                                         int has_draft) {
    if (!draft_sizes_ok(n_seqs, max_draft, n_vocab) || n_seqs == 0 || !known_act(x_type) ||
        (form != Q2_0_DRAFT_LOGITS && form != Q2_0_DRAFT_PROBS))
        return 0;
    return q2_0::draft_plan(n_seqs, max_draft, n_vocab, has_draft != 0, q2_0::act_bytes((q2_0::Act)x_type),
                            form == Q2_0_DRAFT_PROBS).ws_bytes;
}

int q2_0_draft_verify(const void *target, int64_t ld_target, const void *draft, int64_t ld_draft, int x_type, int form,
                      int64_t n_vocab, const float *temperature, const int32_t *tokens, const int32_t *n_draft, const float *u,
                      int64_t n_seqs, int64_t max_draft, int32_t *out, int32_t *n_accepted, void *workspace, size_t ws_bytes,
                      void *stream) {
    if (!draft_sizes_ok(n_seqs, max_draft, n_vocab)) return Q2_0_ERR_SHAPE;
    if (n_seqs == 0) return Q2_0_OK;
    const bool probs = form == Q2_0_DRAFT_PROBS, has_draft = draft != nullptr && max_draft > 0;
    const q2_0::DraftPlan p = q2_0::draft_plan(n_seqs, max_draft, n_vocab, has_draft,
                                               known_act(x_type) ? q2_0::act_bytes((q2_0::Act)x_type) : 4, probs);   // (refused below)
    if (p.stat_groups > kMaxGroups || p.sum_groups > kMaxGroups) return Q2_0_ERR_SHAPE;
    if (!target || !n_draft || !u || !out || !n_accepted || (max_draft > 0 && !tokens)) return Q2_0_ERR_NULL;
    if (ld_target < n_vocab || (has_draft && ld_draft < n_vocab)) return Q2_0_ERR_LAYOUT;
    if (!known_act(x_type) || (form != Q2_0_DRAFT_LOGITS && !probs) || (probs && temperature)) return Q2_0_ERR_UNSUPPORTED;
    const uintptr_t eb = q2_0::act_bytes((q2_0::Act)x_type);
    if (!aligned(target, eb) || !aligned(draft, eb) || !aligned(temperature, 4) || !aligned(tokens, 4) || !aligned(n_draft, 4) ||
        !aligned(u, 4) || !aligned(out, 4) || !aligned(n_accepted, 4))
        return Q2_0_ERR_ALIGN;
    if (ws_bytes < p.ws_bytes || !workspace || !aligned(workspace, 16)) return Q2_0_ERR_WORKSPACE;
    q2_0::DraftVerify a;
    a.target = target, a.draft = has_draft ? draft : nullptr;
    a.ld_target = ld_target, a.ld_draft = ld_draft;
    a.n_vocab = (int)n_vocab, a.n_seqs = (int)n_seqs, a.max_draft = (int)max_draft;
    a.temperature = temperature;
    a.tokens = tokens, a.n_draft = n_draft, a.u = u;
    a.out = out, a.n_accepted = n_accepted;
    a.ws = static_cast<char *>(workspace);
    return q2_0::record_hip_error(q2_0::launch_draft_verify(a, p, (q2_0::Act)x_type, probs, static_cast<hipStream_t>(stream)));
}

int q2_0_kv_copy(const q2_0_kv_cache *to, const q2_0_kv_cache *from, const int32_t *src, const int32_t *dst, int64_t n,
                 void *stream) {
    if (!to || !from) return Q2_0_ERR_NULL;
    if (!cache_shape_ok(*to) || !cache_shape_ok(*from) || !same_pages(*to, *from) || !in(n, 0, kMaxInt) ||
        copy_groups(*to, n) > kMaxGroups)
        return Q2_0_ERR_SHAPE;
    if (n == 0) return Q2_0_OK;
    if (!src || !dst) return Q2_0_ERR_NULL;
    for (const q2_0_kv_cache *c : {to, from}) {
        const int st = check_cache(*c);
        if (st) return st;
    }
    if (!cache_known(*to) || !cache_known(*from) || to->type != from->type) return Q2_0_ERR_UNSUPPORTED;
    if (!cache_aligned(*to) || !cache_aligned(*from) || !aligned(src, 4) || !aligned(dst, 4)) return Q2_0_ERR_ALIGN;
    q2_0::KvCopy a;
    a.to = rows_of(*to), a.from = rows_of(*from);
    a.shape = shape_of(*to);
    a.to_pages = (int)to->n_pages, a.from_pages = (int)from->n_pages;
    a.src = src, a.dst = dst, a.n = (int)n;
    return q2_0::record_hip_error(q2_0::launch_kv_copy(a, static_cast<hipStream_t>(stream)));
}

size_t q2_0_kv_fork_workspace_bytes(int64_t n) { return in(n, 0, kMaxInt) ? (size_t)n * 4 : 0; }

int q2_0_kv_fork(int32_t *ref, int64_t n_pages, int32_t *table, int64_t n_seqs, int64_t table_len, int64_t ld_table,
                 int64_t page_size, int32_t *lens, const int32_t *src, const int32_t *dst, int64_t n, void *workspace,
                 size_t ws_bytes, void *stream) {
    if (!table_ok(n_seqs, table_len) || !in(n_pages, 0, kMaxPages) || !in(page_size, 1, kMaxInt) || !in(n, 0, kMaxInt) ||
        row_groups(n, table_len) > kMaxGroups)
        return Q2_0_ERR_SHAPE;
    if (n == 0 || n_seqs == 0) return Q2_0_OK;
    if ((n_pages > 0 && !ref) || (table_len > 0 && !table) || !lens || !src || !dst) return Q2_0_ERR_NULL;
    if (ld_table < table_len) return Q2_0_ERR_LAYOUT;
    if (!aligned(ref, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(src, 4) || !aligned(dst, 4)) return Q2_0_ERR_ALIGN;
    if (ws_bytes < q2_0_kv_fork_workspace_bytes(n) || !workspace || !aligned(workspace, 16)) return Q2_0_ERR_WORKSPACE;
    q2_0::KvFork a;
    a.t = table_of(table, ld_table, n_seqs, table_len, lens);
    a.page = q2_0::FastDiv::make((uint32_t)page_size);
    a.ref = ref, a.n_pages = (int)n_pages;
    a.src = src, a.dst = dst, a.n = (int)n;
    a.plan = static_cast<int32_t *>(workspace);
    return q2_0::record_hip_error(q2_0::launch_kv_fork(a, static_cast<hipStream_t>(stream)));
}

size_t q2_0_kv_resize_workspace_bytes(int64_t n_seqs, int64_t n_pages) {
    return in(n_seqs, 1, q2_0::kResizeMaxSeqs) && in(n_pages, 0, kMaxPages)
               ? (size_t)n_seqs * 32 + (size_t)n_pages * 4 + (size_t)((n_pages + 31) / 32 + 2) * 4
               : 0;
}

int q2_0_kv_resize(const q2_0_kv_cache *cache, const q2_0_kv_pages *pages, int32_t *table, int64_t n_seqs, int64_t table_len,
                   int64_t ld_table, int32_t *lens, const int32_t *new_lens, int32_t *missing, void *workspace,
                   size_t ws_bytes, void *stream) {
    if (!cache || !pages) return Q2_0_ERR_NULL;
    const q2_0_kv_cache &c = *cache;
    if (!cache_shape_ok(c) || !table_ok(n_seqs, table_len) || n_seqs > q2_0::kResizeMaxSeqs || pages->n_pages != c.n_pages ||
        row_groups(n_seqs, table_len) + copy_groups(c, n_seqs) > kMaxGroups)
        return Q2_0_ERR_SHAPE;
    if (n_seqs == 0) return Q2_0_OK;
    if ((c.n_pages > 0 && (!pages->ref || !pages->free)) || (table_len > 0 && !table) || !lens || !new_lens || !missing)
        return Q2_0_ERR_NULL;
    const int st = check_cache(c);
    if (st) return st;
    if (ld_table < table_len) return Q2_0_ERR_LAYOUT;
    if (!cache_known(c)) return Q2_0_ERR_UNSUPPORTED;
    if (!cache_aligned(c) || !aligned(pages->ref, 4) || !aligned(pages->free, 4) || !aligned(table, 4) || !aligned(lens, 4) ||
        !aligned(new_lens, 4) || !aligned(missing, 4))
        return Q2_0_ERR_ALIGN;
    if (ws_bytes < q2_0_kv_resize_workspace_bytes(n_seqs, c.n_pages) || !workspace || !aligned(workspace, 16))
        return Q2_0_ERR_WORKSPACE;
    q2_0::KvResize a;
    a.t = table_of(table, ld_table, n_seqs, table_len, lens);
    a.rows = rows_of(c);
    a.shape = shape_of(c);
    a.ref = pages->ref, a.free = pages->free, a.n_pages = (int)c.n_pages;
    a.new_lens = new_lens, a.missing = missing;
    a.plan = static_cast<int32_t *>(workspace);
    a.fresh = a.plan + n_seqs * 8;
    a.before = a.fresh + c.n_pages;
    return q2_0::record_hip_error(q2_0::launch_kv_resize(a, static_cast<hipStream_t>(stream)));
}

size_t q2_0_kv_compact_workspace_bytes(int64_t n_pages) {
    return in(n_pages, 1, kMaxPages) ? (size_t)((n_pages + 31) / 32) * 4 : 0;
}

int q2_0_kv_compact(const q2_0_kv_cache *to, const q2_0_kv_pages *to_pages, const q2_0_kv_cache *from,
                    const q2_0_kv_pages *from_pages, const int32_t *table, int64_t n_seqs, int64_t table_len, int64_t ld_table,
                    const int32_t *lens, int32_t *to_table, int64_t ld_to_table, int32_t *n_used, void *workspace,
                    size_t ws_bytes, void *stream) {
    if (!to || !from || !to_pages || !from_pages) return Q2_0_ERR_NULL;
    if (!cache_shape_ok(*to) || !cache_shape_ok(*from) || !same_pages(*to, *from) || !table_ok(n_seqs, table_len) ||
        to_pages->n_pages != to->n_pages || from_pages->n_pages != from->n_pages ||
        row_groups(n_seqs, table_len) + copy_groups(*from, from->n_pages) + (to->n_pages + 255) / 256 > kMaxGroups)
        return Q2_0_ERR_SHAPE;
    const bool rows = n_seqs > 0 && table_len > 0;
    if (!n_used || (from->n_pages > 0 && (!from_pages->ref || !from_pages->free)) ||
        (to->n_pages > 0 && (!to_pages->ref || !to_pages->free)) || (rows && (!table || !lens || !to_table)))
        return Q2_0_ERR_NULL;
    for (const q2_0_kv_cache *c : {to, from}) {
        const int st = check_cache(*c);
        if (st) return st;
    }
    // all of it moves at once: nothing of the one pool may be the other's
    if (ld_table < table_len || ld_to_table < table_len || to->k == from->k || to->v == from->v || to->k == from->v ||
        to->v == from->k || (to->n_pages > 0 && (to_pages->ref == from_pages->ref || to_pages->free == from_pages->free)) ||
        (rows && table == to_table))
        return Q2_0_ERR_LAYOUT;
    if (!cache_known(*to) || !cache_known(*from) || to->type != from->type) return Q2_0_ERR_UNSUPPORTED;
    for (const q2_0_kv_pages *p : {to_pages, from_pages})
        if (!aligned(p->ref, 4) || !aligned(p->free, 4)) return Q2_0_ERR_ALIGN;
    if (!cache_aligned(*to) || !cache_aligned(*from) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(to_table, 4) ||
        !aligned(n_used, 4))
        return Q2_0_ERR_ALIGN;
    const size_t need = q2_0_kv_compact_workspace_bytes(from->n_pages);
    if (need && (ws_bytes < need || !workspace || !aligned(workspace, 16))) return Q2_0_ERR_WORKSPACE;
    q2_0::KvCompact a;
    a.t = table_of(table, ld_table, n_seqs, rows ? table_len : 0, lens);
    a.to = rows_of(*to), a.from = rows_of(*from);
    a.shape = shape_of(*to);
    a.ref = from_pages->ref, a.free = from_pages->free;
    a.from_pages = (int)from->n_pages, a.to_pages = (int)to->n_pages;
    a.to_ref = to_pages->ref, a.to_free = to_pages->free;
    a.to_table = to_table, a.ld_to = ld_to_table;
    a.n_used = n_used;
    a.before = static_cast<int32_t *>(workspace);
    return q2_0::record_hip_error(q2_0::launch_kv_compact(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
