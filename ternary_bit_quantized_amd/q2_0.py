"""Python binding of libq2_0.so (ctypes).  Argument marshalling only.

Every computation happens in the HIP kernels behind the C ABI declared in
include/q2_0.h.  PyTorch supplies device memory and the current stream; there is
no fallback of any kind: if the library is missing or a call fails, an exception
is raised.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# Q2_0_LIB names another build of the library (the sanitized host-only build of
# ternary_bit_quantized_amd.build --sanitize, for the ABI tests); default: the in-tree one.
LIB_PATH = os.environ.get("Q2_0_LIB") or os.path.join(PKG, "libq2_0.so")

Q2_0_OK = 0
Q2_0_ERR_NULL = 1
Q2_0_ERR_SHAPE = 2
Q2_0_ERR_LAYOUT = 3
Q2_0_ERR_ALIGN = 4
Q2_0_ERR_UNSUPPORTED = 5
Q2_0_ERR_WORKSPACE = 6
Q2_0_ERR_HIP = 7
Q2_0_ERR_TOO_LARGE = 8
Q2_0_PREC_F16_MFMA = 0
Q2_0_PREC_F32 = 1
Q2_0_PREC_F32_MFMA = 2
Q2_0_ACT_F32 = 0
Q2_0_ACT_F16 = 1
Q2_0_ACT_BF16 = 2
Q2_0_ROPE_HALF = 0
Q2_0_ROPE_PAIRS = 1
Q2_0_SCORE_SOFTMAX = 0
Q2_0_SCORE_SIGMOID = 1
Q2_0_DRAFT_LOGITS = 0
Q2_0_DRAFT_PROBS = 1
BLOCK_WEIGHTS = 64
BLOCK_BYTES = 18
MAT_VEC_MAX_N = 8
NOALLOC_SCRATCH_BYTES = 64 << 20
ATTN_MAX_QT = 16
MOE_LAYER_MAX_TOKENS = 64
MOE_LAYER_MAX_USED = 32
DRAFT_MAX = 15

EXPORTS = ("q2_0_get_rows", "q2_0_mul_mat_vec", "q2_0_mul_mat_vec_group", "q2_0_mul_mat",
           "q2_0_mul_mat_workspace_bytes", "q2_0_mul_mat_group", "q2_0_mul_mat_group_workspace_bytes",
           "q2_0_mul_mat_vec_act", "q2_0_mul_mat_vec_group_act", "q2_0_mul_mat_act", "q2_0_mul_mat_group_act",
           "q2_0_quantize", "q2_0_repack_g128", "q2_0_mul_mat_id", "q2_0_mul_mat_id_workspace_bytes",
           "q2_0_mul_mat_noalloc", "q2_0_mul_mat_vec_batch", "q2_0_kv_append", "q2_0_attn_shared",
           "q2_0_attn_shared_workspace_bytes", "q2_0_moe_route", "q2_0_moe_layer", "q2_0_moe_layer_workspace_bytes",
           "q2_0_moe_route_groups", "q2_0_draft_verify", "q2_0_draft_verify_workspace_bytes", "q2_0_kv_copy",
           "q2_0_kv_fork", "q2_0_kv_fork_workspace_bytes", "q2_0_kv_resize", "q2_0_kv_resize_workspace_bytes",
           "q2_0_kv_compact", "q2_0_kv_compact_workspace_bytes",
           "q2_0_status_string", "q2_0_last_hip_error", "q2_0_version")


class MatVecItem(ctypes.Structure):
    """q2_0_mat_vec_item: one matrix of a grouped mat-vec."""
    _fields_ = [("w", ctypes.c_void_p), ("M", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64)]


class MatVecBatchItem(ctypes.Structure):
    """q2_0_mat_vec_batch_item: one product of a batched mat-vec (its own K and x)."""
    _fields_ = [("w", ctypes.c_void_p), ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class KvCache(ctypes.Structure):
    """q2_0_kv_cache: the two pools of a paged key/value cache; strides in elements."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("n_kv", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class KvPages(ctypes.Structure):
    """q2_0_kv_pages: counts and free bits of a cache's pages."""
    _fields_ = [("ref", ctypes.c_void_p), ("free", ctypes.c_void_p), ("n_pages", ctypes.c_int64)]


def make_batch_items(entries):
    """[(w_ptr, M, K, x_ptr, ldx, y_ptr, ldy), ...] -> a ctypes array for mul_mat_vec_batch_raw."""
    arr = (MatVecBatchItem * len(entries))()
    for i, e in enumerate(entries):
        arr[i] = MatVecBatchItem(*e)
    return arr


def make_items(entries):
    """[(w_ptr, M, y_ptr, ldy), ...] -> a ctypes array to pass to mul_mat_vec_group_raw."""
    arr = (MatVecItem * len(entries))()
    for i, (w, M, y, ldy) in enumerate(entries):
        arr[i] = MatVecItem(w, M, y, ldy)
    return arr


class Q2_0Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().q2_0_status_string(status).decode()
        if status == Q2_0_ERR_HIP:
            msg += " (hipError %d)" % lib().q2_0_last_hip_error()
        super().__init__("%s: %s" % (what, msg))


_lib = None


def lib() -> ctypes.CDLL:
    """Load libq2_0.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libq2_0.so is not built (%s); run `python -m "
                               "ternary_bit_quantized_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I64 = ctypes.c_void_p, ctypes.c_int64
        L.q2_0_get_rows.argtypes = [P, I64, I64, P, I64, P, I64, P]
        L.q2_0_mul_mat_vec.argtypes = [P, I64, I64, P, I64, I64, P, I64, P]
        L.q2_0_mul_mat_vec_group.argtypes = [P, I64, I64, P, I64, I64, P]
        L.q2_0_mul_mat_vec_group.restype = ctypes.c_int
        L.q2_0_mul_mat.argtypes = [P, I64, I64, P, I64, I64, P, I64, ctypes.c_int, P,
                                   ctypes.c_size_t, P]
        L.q2_0_mul_mat_workspace_bytes.argtypes = [I64, I64, I64, ctypes.c_int]
        L.q2_0_mul_mat_workspace_bytes.restype = ctypes.c_size_t
        L.q2_0_mul_mat_group.argtypes = [P, I64, I64, P, I64, I64, ctypes.c_int, P, ctypes.c_size_t, P]
        L.q2_0_mul_mat_group.restype = ctypes.c_int
        L.q2_0_mul_mat_group_workspace_bytes.argtypes = [P, I64, I64, I64, ctypes.c_int]
        L.q2_0_mul_mat_group_workspace_bytes.restype = ctypes.c_size_t
        C = ctypes.c_int
        L.q2_0_mul_mat_vec_act.argtypes = [P, I64, I64, P, C, I64, I64, P, I64, P]
        L.q2_0_mul_mat_vec_group_act.argtypes = [P, I64, I64, P, C, I64, I64, P]
        L.q2_0_mul_mat_act.argtypes = [P, I64, I64, P, C, I64, I64, P, I64, C, P, ctypes.c_size_t, P]
        L.q2_0_mul_mat_group_act.argtypes = [P, I64, I64, P, C, I64, I64, C, P, ctypes.c_size_t, P]
        L.q2_0_quantize.argtypes = [P, I64, I64, I64, P, P]
        L.q2_0_mul_mat_id.argtypes = [P, I64, I64, I64, P, C, I64, I64, P, I64, I64, P, I64, C, P,
                                      ctypes.c_size_t, P]
        L.q2_0_mul_mat_id_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, C]
        L.q2_0_mul_mat_id_workspace_bytes.restype = ctypes.c_size_t
        L.q2_0_repack_g128.argtypes = [P, I64, I64, P, P]
        L.q2_0_mul_mat_vec_batch.argtypes = [P, I64, ctypes.c_int, I64, P]
        L.q2_0_mul_mat_vec_batch.restype = ctypes.c_int
        L.q2_0_mul_mat_noalloc.argtypes = [P, I64, I64, P, I64, I64, P, I64, ctypes.c_int, P]
        L.q2_0_mul_mat_noalloc.restype = ctypes.c_int
        L.q2_0_kv_append.argtypes = [P, P, I64, I64, I64, P, P, I64, P, I64, I64, P, I64, P, I64, C, P, I64, I64, C, P,
                                     I64, P]
        L.q2_0_kv_append.restype = C
        L.q2_0_attn_shared.argtypes = [P, P, I64, I64, I64, P, I64, I64, P, I64, I64, I64, ctypes.c_float, P, I64, P,
                                       ctypes.c_size_t, P]
        L.q2_0_attn_shared.restype = C
        L.q2_0_attn_shared_workspace_bytes.argtypes = [I64] * 7
        L.q2_0_attn_shared_workspace_bytes.restype = ctypes.c_size_t
        L.q2_0_moe_route.argtypes = [P, C, I64, I64, I64, I64, C, P, P, P]
        L.q2_0_moe_route.restype = C
        L.q2_0_moe_layer.argtypes = [P, P, P, I64, I64, I64, P, C, I64, P, P, I64, I64, P, I64, P, ctypes.c_size_t, P]
        L.q2_0_moe_layer.restype = C
        L.q2_0_moe_layer_workspace_bytes.argtypes = [I64] * 4
        L.q2_0_moe_layer_workspace_bytes.restype = ctypes.c_size_t
        S = ctypes.c_size_t
        L.q2_0_moe_route_groups.argtypes = [P, C, I64, I64, I64, I64, C, P, I64, I64, I64, C, ctypes.c_float, P, P, P]
        L.q2_0_draft_verify.argtypes = [P, I64, P, I64, C, C, I64, P, P, P, P, I64, I64, P, P, P, S, P]
        L.q2_0_draft_verify_workspace_bytes.argtypes = [I64, I64, I64, C, C, C]
        L.q2_0_kv_copy.argtypes = [P, P, P, P, I64, P]
        L.q2_0_kv_fork.argtypes = [P, I64, P, I64, I64, I64, I64, P, P, P, I64, P, S, P]
        L.q2_0_kv_fork_workspace_bytes.argtypes = [I64]
        L.q2_0_kv_resize.argtypes = [P, P, P, I64, I64, I64, P, P, P, P, S, P]
        L.q2_0_kv_resize_workspace_bytes.argtypes = [I64, I64]
        L.q2_0_kv_compact.argtypes = [P, P, P, P, P, I64, I64, I64, P, P, I64, P, P, S, P]
        L.q2_0_kv_compact_workspace_bytes.argtypes = [I64]
        for f in (L.q2_0_moe_route_groups, L.q2_0_draft_verify, L.q2_0_kv_copy, L.q2_0_kv_fork, L.q2_0_kv_resize,
                  L.q2_0_kv_compact):
            f.restype = C
        for f in (L.q2_0_draft_verify_workspace_bytes, L.q2_0_kv_fork_workspace_bytes, L.q2_0_kv_resize_workspace_bytes,
                  L.q2_0_kv_compact_workspace_bytes):
            f.restype = S
        for f in (L.q2_0_mul_mat_vec_act, L.q2_0_mul_mat_vec_group_act, L.q2_0_mul_mat_act,
                  L.q2_0_mul_mat_group_act, L.q2_0_quantize, L.q2_0_repack_g128, L.q2_0_mul_mat_id):
            f.restype = ctypes.c_int
        L.q2_0_status_string.argtypes = [ctypes.c_int]
        L.q2_0_status_string.restype = ctypes.c_char_p
        L.q2_0_version.restype = ctypes.c_char_p
        for f in (L.q2_0_get_rows, L.q2_0_mul_mat_vec, L.q2_0_mul_mat, L.q2_0_last_hip_error):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, what: str) -> None:
    if status != Q2_0_OK:
        raise Q2_0Error(status, what)


# ----------------------------------------------------------------------------- raw (pointers)

def _items_ptr(items):
    return ctypes.cast(items, ctypes.c_void_p) if items is not None else None


def get_rows_raw(w: int, M: int, K: int, ids: int, n_ids: int, out: int, ld_out: int,
                 stream: int = 0) -> int:
    return lib().q2_0_get_rows(w, M, K, ids, n_ids, out, ld_out, stream)


def mul_mat_vec_raw(w: int, M: int, K: int, x: int, ldx: int, N: int, y: int, ldy: int,
                    stream: int = 0) -> int:
    return lib().q2_0_mul_mat_vec(w, M, K, x, ldx, N, y, ldy, stream)


def mul_mat_vec_group_raw(items, n_items: int, K: int, x: int, ldx: int, N: int,
                          stream: int = 0) -> int:
    """items: a ctypes array from make_items (or None with n_items == 0)."""
    return lib().q2_0_mul_mat_vec_group(ctypes.cast(items, ctypes.c_void_p) if items is not None else None,
                                        n_items, K, x, ldx, N, stream)


def mul_mat_vec_batch_raw(items, n_items: int, x_type: int, N: int, stream: int = 0) -> int:
    """items: a ctypes array from make_batch_items (or None with n_items == 0)."""
    return lib().q2_0_mul_mat_vec_batch(_items_ptr(items), n_items, x_type, N, stream)


def mul_mat_raw(w: int, M: int, K: int, x: int, ldx: int, N: int, y: int, ldy: int, precision: int,
                workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_mul_mat(w, M, K, x, ldx, N, y, ldy, precision, workspace, ws_bytes, stream)


def mul_mat_noalloc_raw(w: int, M: int, K: int, x: int, ldx: int, N: int, y: int, ldy: int, precision: int,
                        stream: int = 0) -> int:
    return lib().q2_0_mul_mat_noalloc(w, M, K, x, ldx, N, y, ldy, precision, stream)


def mul_mat_workspace_bytes(M: int, K: int, N: int, precision: int) -> int:
    return int(lib().q2_0_mul_mat_workspace_bytes(M, K, N, precision))


def mul_mat_group_raw(items, n_items: int, K: int, x: int, ldx: int, N: int, precision: int,
                      workspace: int, ws_bytes: int, stream: int = 0) -> int:
    """items: a ctypes array from make_items (or None with n_items == 0)."""
    return lib().q2_0_mul_mat_group(_items_ptr(items), n_items, K, x, ldx, N, precision, workspace, ws_bytes,
                                    stream)


def mul_mat_group_workspace_bytes(items, n_items: int, K: int, N: int, precision: int) -> int:
    return int(lib().q2_0_mul_mat_group_workspace_bytes(_items_ptr(items), n_items, K, N, precision))


def mul_mat_vec_act_raw(w: int, M: int, K: int, x: int, x_type: int, ldx: int, N: int, y: int, ldy: int,
                        stream: int = 0) -> int:
    return lib().q2_0_mul_mat_vec_act(w, M, K, x, x_type, ldx, N, y, ldy, stream)


def mul_mat_vec_group_act_raw(items, n_items: int, K: int, x: int, x_type: int, ldx: int, N: int,
                              stream: int = 0) -> int:
    return lib().q2_0_mul_mat_vec_group_act(_items_ptr(items), n_items, K, x, x_type, ldx, N, stream)


def mul_mat_act_raw(w: int, M: int, K: int, x: int, x_type: int, ldx: int, N: int, y: int, ldy: int,
                    precision: int, workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_mul_mat_act(w, M, K, x, x_type, ldx, N, y, ldy, precision, workspace, ws_bytes, stream)


def mul_mat_group_act_raw(items, n_items: int, K: int, x: int, x_type: int, ldx: int, N: int, precision: int,
                          workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_mul_mat_group_act(_items_ptr(items), n_items, K, x, x_type, ldx, N, precision,
                                        workspace, ws_bytes, stream)


def mul_mat_id_raw(w: int, n_expert: int, M: int, K: int, x: int, x_type: int, ldx: int, x_slots: int,
                   ids: int, n_used: int, n_tokens: int, y: int, ldy: int, precision: int, workspace: int,
                   ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_mul_mat_id(w, n_expert, M, K, x, x_type, ldx, x_slots, ids, n_used, n_tokens, y, ldy,
                                 precision, workspace, ws_bytes, stream)


def mul_mat_id_workspace_bytes(n_expert: int, M: int, K: int, n_used: int, n_tokens: int, precision: int) -> int:
    return int(lib().q2_0_mul_mat_id_workspace_bytes(n_expert, M, K, n_used, n_tokens, precision))


def quantize_raw(src: int, M: int, K: int, ld_src: int, w: int, stream: int = 0) -> int:
    return lib().q2_0_quantize(src, M, K, ld_src, w, stream)


def repack_g128_raw(w128: int, M: int, K: int, w: int, stream: int = 0) -> int:
    return lib().q2_0_repack_g128(w128, M, K, w, stream)


def kv_append_raw(cache: KvCache, table: int, n_seqs: int, table_len: int, ld_table: int, seq: int, pos: int,
                  n_tokens: int, q: int, ldq: int, n_q: int, k: int, ldk: int, v: int, ldv: int, x_type: int, rope: int,
                  n_pos: int, rot_dim: int, style: int, q_out: int, ldqo: int, stream: int = 0) -> int:
    return lib().q2_0_kv_append(ctypes.byref(cache) if cache is not None else None, table, n_seqs, table_len, ld_table,
                                seq, pos, n_tokens, q, ldq, n_q, k, ldk, v, ldv, x_type, rope, n_pos, rot_dim, style,
                                q_out, ldqo, stream)


def attn_shared_raw(cache: KvCache, table: int, n_seqs: int, table_len: int, ld_table: int, lens: int, prefix_len: int,
                    max_len: int, q: int, ldq: int, n_q: int, n_qt: int, scale: float, out: int, ldo: int,
                    workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_attn_shared(ctypes.byref(cache) if cache is not None else None, table, n_seqs, table_len, ld_table,
                                  lens, prefix_len, max_len, q, ldq, n_q, n_qt, scale, out, ldo, workspace, ws_bytes,
                                  stream)


@functools.lru_cache(maxsize=1024)      # (a function of the sizes alone)
def attn_shared_workspace_bytes(n_seqs: int, n_q: int, n_kv: int, head_dim: int, n_qt: int, prefix_len: int,
                                max_len: int) -> int:
    return lib().q2_0_attn_shared_workspace_bytes(n_seqs, n_q, n_kv, head_dim, n_qt, prefix_len, max_len)


def moe_route_raw(logits: int, x_type: int, ld: int, n_tokens: int, n_expert: int, n_used: int, normalise: int, ids: int,
                  weights: int, stream: int = 0) -> int:
    return lib().q2_0_moe_route(logits, x_type, ld, n_tokens, n_expert, n_used, normalise, ids, weights, stream)


def moe_layer_raw(w_gate: int, w_up: int, w_down: int, n_expert: int, n_ff: int, K: int, x: int, x_type: int, ldx: int,
                  ids: int, weights: int, n_used: int, n_tokens: int, y: int, ldy: int, workspace: int, ws_bytes: int,
                  stream: int = 0) -> int:
    return lib().q2_0_moe_layer(w_gate, w_up, w_down, n_expert, n_ff, K, x, x_type, ldx, ids, weights, n_used, n_tokens,
                                y, ldy, workspace, ws_bytes, stream)


@functools.lru_cache(maxsize=1024)      # (a function of the sizes alone)
def moe_layer_workspace_bytes(n_ff: int, K: int, n_used: int, n_tokens: int) -> int:
    return lib().q2_0_moe_layer_workspace_bytes(n_ff, K, n_used, n_tokens)


def moe_route_groups_raw(logits: int, x_type: int, ld: int, n_tokens: int, n_expert: int, n_used: int, score: int, bias: int,
                         n_group: int, n_group_used: int, group_top: int, normalise: int, scale: float, ids: int,
                         weights: int, stream: int = 0) -> int:
    return lib().q2_0_moe_route_groups(logits, x_type, ld, n_tokens, n_expert, n_used, score, bias, n_group, n_group_used,
                                       group_top, normalise, scale, ids, weights, stream)


def draft_verify_raw(target: int, ld_target: int, draft: int, ld_draft: int, x_type: int, form: int, n_vocab: int,
                     temperature: int, tokens: int, n_draft: int, u: int, n_seqs: int, max_draft: int, out: int,
                     n_accepted: int, workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_draft_verify(target, ld_target, draft, ld_draft, x_type, form, n_vocab, temperature, tokens, n_draft, u,
                                   n_seqs, max_draft, out, n_accepted, workspace, ws_bytes, stream)


@functools.lru_cache(maxsize=1024)      # (a function of the sizes alone)
def draft_verify_workspace_bytes(n_seqs: int, max_draft: int, n_vocab: int, x_type: int, form: int, has_draft: int) -> int:
    return lib().q2_0_draft_verify_workspace_bytes(n_seqs, max_draft, n_vocab, x_type, form, has_draft)


def _ref(struct):
    return ctypes.byref(struct) if struct is not None else None


def kv_copy_raw(to: KvCache, frm: KvCache, src: int, dst: int, n: int, stream: int = 0) -> int:
    return lib().q2_0_kv_copy(_ref(to), _ref(frm), src, dst, n, stream)


def kv_fork_raw(ref: int, n_pages: int, table: int, n_seqs: int, table_len: int, ld_table: int, page_size: int, lens: int,
                src: int, dst: int, n: int, workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_kv_fork(ref, n_pages, table, n_seqs, table_len, ld_table, page_size, lens, src, dst, n, workspace,
                              ws_bytes, stream)


@functools.lru_cache(maxsize=1024)      # (a function of the sizes alone)
def kv_fork_workspace_bytes(n: int) -> int:
    return lib().q2_0_kv_fork_workspace_bytes(n)


def kv_resize_raw(cache: KvCache, pages: KvPages, table: int, n_seqs: int, table_len: int, ld_table: int, lens: int,
                  new_lens: int, missing: int, workspace: int, ws_bytes: int, stream: int = 0) -> int:
    return lib().q2_0_kv_resize(_ref(cache), _ref(pages), table, n_seqs, table_len, ld_table, lens, new_lens, missing,
                                workspace, ws_bytes, stream)


@functools.lru_cache(maxsize=1024)      # (a function of the sizes alone)
def kv_resize_workspace_bytes(n_seqs: int, n_pages: int) -> int:
    return lib().q2_0_kv_resize_workspace_bytes(n_seqs, n_pages)


def kv_compact_raw(to: KvCache, to_pages: KvPages, frm: KvCache, from_pages: KvPages, table: int, n_seqs: int, table_len: int,
                   ld_table: int, lens: int, to_table: int, ld_to_table: int, n_used: int, workspace: int, ws_bytes: int,
                   stream: int = 0) -> int:
    return lib().q2_0_kv_compact(_ref(to), _ref(to_pages), _ref(frm), _ref(from_pages), table, n_seqs, table_len, ld_table,
                                 lens, to_table, ld_to_table, n_used, workspace, ws_bytes, stream)


@functools.lru_cache(maxsize=1024)      # (a function of the sizes alone)
def kv_compact_workspace_bytes(n_pages: int) -> int:
    return lib().q2_0_kv_compact_workspace_bytes(n_pages)


def version() -> str:
    return lib().q2_0_version().decode()


# ----------------------------------------------------------------------------- torch tensors

def _stream(stream, dev=None):
    import torch
    if stream is None:      # the current stream's handle, without the Stream object around it (2.8 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    if dev is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError("stream must be one of the current device")
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _other(stream):
    """A call's stream as torch has it; None where that is the current one."""
    import torch
    handle = _stream(stream)
    if handle == torch.cuda.current_stream().cuda_stream:
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()      # (0 is the default stream)


def _empty(like, shape, dtype, stream, result=True):
    """A new tensor on like's device for a call whose kernels run on `stream`.  Its memory is that stream's: what the
    allocator gives and takes back is in order with the kernels, though another stream is current.  The caller may
    read a result on the current stream and free it then, so the allocator is told of that one too."""
    other = None if stream is None else _other(stream)
    if other is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    with torch.cuda.stream(other):
        t = like.new_empty(shape, dtype=dtype)
    if result:
        t.record_stream(torch.cuda.current_stream())
    return t


def _cols(t, K, name):
    """A (N, >=K) float32 device tensor with unit column stride -> (ptr, N, ld)."""
    import torch
    if t.dtype != torch.float32 or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("%s must be a 2-D float32 CUDA tensor with unit inner stride" % name)
    if t.shape[1] < K:
        raise ValueError("%s must have at least %d columns" % (name, K))
    ld = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])
    return t.data_ptr(), t.shape[0], ld


def _xcols(t, K, name):
    """An activation tensor (N, >=K) of float32, float16 or bfloat16 with unit inner stride
    -> (ptr, N, ld, x_type)."""
    import torch
    types = {torch.float32: Q2_0_ACT_F32, torch.float16: Q2_0_ACT_F16, torch.bfloat16: Q2_0_ACT_BF16}
    if t.dtype not in types or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("%s must be a 2-D float32/float16/bfloat16 CUDA tensor with unit inner stride" % name)
    if t.shape[1] < K:
        raise ValueError("%s must have at least %d columns" % (name, K))
    ld = t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])
    return t.data_ptr(), t.shape[0], ld, types[t.dtype]


def q2_0_mul_mat_id(w, n_expert: int, M: int, K: int, x, ids, precision: int = Q2_0_PREC_F16_MFMA, y=None,
                    workspace=None, stream=None):
    """Expert product: w holds n_expert (M, K) Q2_0 matrices back to back; ids (n_tokens, n_used)
    int32 on the device; x (n_tokens * x_slots, K) with x_slots 1 or n_used.  Returns
    y (n_tokens * n_used, M) float32, row t * n_used + u = W_{ids[t, u]} x[t * x_slots + u % x_slots]."""
    import torch
    if ids.dtype != torch.int32 or not ids.is_contiguous() or ids.dim() != 2:
        raise ValueError("ids must be a contiguous 2-D int32 tensor")
    n_tokens, n_used = ids.shape
    xp, rows, ldx, xt = _xcols(x, K, "x")
    if rows != n_tokens and rows != n_tokens * n_used:
        raise ValueError("x must have n_tokens or n_tokens * n_used rows")
    x_slots = 1 if rows == n_tokens else n_used
    if y is None:
        y = _empty(x, (n_tokens * n_used, M), torch.float32, stream)
    yp, _, ldy = _cols(y, M, "y")
    need = mul_mat_id_workspace_bytes(n_expert, M, K, n_used, n_tokens, precision)
    if workspace is None:
        workspace = _empty(x, max(need, 16), torch.uint8, stream, result=False)
    wsb = workspace.numel() * workspace.element_size()
    _check(mul_mat_id_raw(w.data_ptr(), n_expert, M, K, xp, xt, ldx, x_slots, ids.data_ptr(), n_used, n_tokens,
                          yp, ldy, precision, workspace.data_ptr(), wsb, _stream(stream)), "q2_0_mul_mat_id")
    return y


def q2_0_quantize(src, w=None, stream=None):
    """Q2_0 (uint8 device tensor (M, K/64*18)) of the float32 weights src (M, K) by the reference quantizer."""
    import torch
    M, K = src.shape
    ptr, _, ld = _cols(src, K, "src")
    if w is None:
        w = _empty(src, (M, K // BLOCK_WEIGHTS * BLOCK_BYTES), torch.uint8, stream)
    _check(quantize_raw(ptr, M, K, ld, w.data_ptr(), _stream(stream)), "q2_0_quantize")
    return w


def q2_0_repack_g128(w128, M: int, K: int, w=None, stream=None):
    """The group-64 Q2_0 tensor of a legacy group-128 tensor w128 (uint8, M rows of K/128*34 bytes)."""
    import torch
    if w is None:
        w = _empty(w128, (M, K // BLOCK_WEIGHTS * BLOCK_BYTES), torch.uint8, stream)
    _check(repack_g128_raw(w128.data_ptr(), M, K, w.data_ptr(), _stream(stream)), "q2_0_repack_g128")
    return w


def q2_0_get_rows(w, M: int, K: int, ids, out=None, stream=None):
    """out[r, :K] = dequantized row ids[r] of the (M, K) Q2_0 matrix w (uint8 device tensor)."""
    import torch
    n = ids.numel()
    if out is None:
        out = _empty(w, (n, K), torch.float32, stream)
    ptr, rows, ld = _cols(out, K, "out")
    if ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 tensor")
    _check(get_rows_raw(w.data_ptr(), M, K, ids.data_ptr(), n, ptr, ld, _stream(stream)),
           "q2_0_get_rows")
    return out


def q2_0_mul_mat_vec(w, M: int, K: int, x, y=None, stream=None):
    """y (N, M) = W x for x (N, K) of float32, float16 or bfloat16, N <= 8; y is float32."""
    import torch
    xp, N, ldx, xt = _xcols(x, K, "x")
    if y is None:
        y = _empty(x, (N, M), torch.float32, stream)
    yp, _, ldy = _cols(y, M, "y")
    _check(mul_mat_vec_act_raw(w.data_ptr(), M, K, xp, xt, ldx, N, yp, ldy, _stream(stream)),
           "q2_0_mul_mat_vec_act")
    return y


def q2_0_mul_mat_vec_group(mats, K: int, x, ys=None, stream=None):
    """mats: [(w, M), ...] sharing K; returns [y_i (N, M_i)] with y_i = W_i x (x float32, float16
    or bfloat16)."""
    import torch
    xp, N, ldx, xt = _xcols(x, K, "x")
    if ys is None:
        ys = [_empty(x, (N, M), torch.float32, stream) for (_, M) in mats]
    entries = []
    for (w, M), y in zip(mats, ys):
        yp, _, ldy = _cols(y, M, "y")
        entries.append((w.data_ptr(), M, yp, ldy))
    items = make_items(entries)
    _check(mul_mat_vec_group_act_raw(items, len(entries), K, xp, xt, ldx, N, _stream(stream)),
           "q2_0_mul_mat_vec_group_act")
    return ys


def q2_0_mul_mat_vec_batch(products, x_type_tensor=None, ys=None, stream=None):
    """products: [(w, M, K, x), ...] with x (N, >=K) device tensors of one dtype (float32,
    float16 or bfloat16) and the same N; returns [y_i (N, M_i) float32] with y_i = W_i x_i."""
    import torch
    entries, out = [], []
    xt0, N0 = None, None
    for i, (w, M, K, x) in enumerate(products):
        xp, N, ldx, xt = _xcols(x, K, "x")
        if xt0 is None:
            xt0, N0 = xt, N
        elif xt != xt0 or N != N0:
            raise ValueError("every x of a batch must have the same dtype and column count")
        y = ys[i] if ys is not None else _empty(x, (N, M), torch.float32, stream)
        yp, _, ldy = _cols(y, M, "y")
        entries.append((w.data_ptr(), M, K, xp, ldx, yp, ldy))
        out.append(y)
    items = make_batch_items(entries)
    _check(mul_mat_vec_batch_raw(items, len(entries), xt0 if xt0 is not None else Q2_0_ACT_F32, N0 or 0,
                                 _stream(stream)), "q2_0_mul_mat_vec_batch")
    return out


def q2_0_mul_mat(w, M: int, K: int, x, precision: int = Q2_0_PREC_F16_MFMA, y=None, workspace=None,
                 stream=None):
    """y (N, M) = W x for x (N, K) of float32, float16 or bfloat16, any N; y is float32."""
    import torch
    xp, N, ldx, xt = _xcols(x, K, "x")
    if y is None:
        y = _empty(x, (N, M), torch.float32, stream)
    yp, _, ldy = _cols(y, M, "y")
    need = mul_mat_workspace_bytes(M, K, N, precision)
    if workspace is None and need:
        workspace = _empty(x, need, torch.uint8, stream, result=False)
    wsp = workspace.data_ptr() if workspace is not None else 0
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(mul_mat_act_raw(w.data_ptr(), M, K, xp, xt, ldx, N, yp, ldy, precision, wsp, wsb, _stream(stream)),
           "q2_0_mul_mat_act")
    return y


def q2_0_mul_mat_group(mats, K: int, x, precision: int = Q2_0_PREC_F16_MFMA, ys=None, workspace=None,
                       stream=None):
    """mats: [(w, M), ...] sharing K; returns [y_i (N, M_i)] with y_i = W_i x, any N (x float32,
    float16 or bfloat16)."""
    import torch
    xp, N, ldx, xt = _xcols(x, K, "x")
    if ys is None:
        ys = [_empty(x, (N, M), torch.float32, stream) for (_, M) in mats]
    entries = []
    for (w, M), y in zip(mats, ys):
        yp, _, ldy = _cols(y, M, "y")
        entries.append((w.data_ptr(), M, yp, ldy))
    items = make_items(entries)
    need = mul_mat_group_workspace_bytes(items, len(entries), K, N, precision)
    if workspace is None and need:
        workspace = _empty(x, need, torch.uint8, stream, result=False)
    wsp = workspace.data_ptr() if workspace is not None else 0
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(mul_mat_group_act_raw(items, len(entries), K, xp, xt, ldx, N, precision, wsp, wsb, _stream(stream)),
           "q2_0_mul_mat_group_act")
    return ys


# ------------------------------------------------------------- decoder-step operators (torch)

@functools.lru_cache(maxsize=None)
def _act_types():
    import torch
    return {torch.float32: Q2_0_ACT_F32, torch.float16: Q2_0_ACT_F16, torch.bfloat16: Q2_0_ACT_BF16}


# These calls launch on the current device, dev: every tensor has to be there (get_device() of a CPU tensor is -1).

def _rows(t, rows, cols, name, dev):
    """A 2-D tensor of `rows` rows of at least `cols` elements, unit inner stride -> row stride."""
    if t.get_device() == dev and t.dim() == 2:
        (n, c), (ld, inner) = t.shape, t.stride()
        if n == rows and c >= cols and (inner == 1 or c <= 1):
            return ld if rows > 1 else max(ld, c)
    raise ValueError("%s must be a 2-D tensor on the current CUDA device of %d rows of at least %d elements with unit "
                     "inner stride" % (name, rows, cols))


def _dense(t, dtype, shape, name, dev):
    if t.dtype != dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on the current CUDA device"
                         % (name, str(dtype).split(".")[-1], tuple(shape)))
    return t.data_ptr()


def _wide(t, name):
    """Columns of a 2-D tensor."""
    if t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % name)
    return t.shape[1]


def _work(workspace, need, like, stream, dev):
    """The workspace given, or one of `need` bytes -> (tensor or None, address, bytes)."""
    if workspace is None:
        if not need:
            return None, 0, 0
        import torch
        workspace = _empty(like, need, torch.uint8, stream, result=False)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _table(t, dev):
    import torch
    if t.dtype == torch.int32 and t.get_device() == dev and t.dim() == 2:
        (n, cols), (ld, inner) = t.shape, t.stride()
        if inner == 1 or cols <= 1:
            return t.data_ptr(), n, cols, ld if n > 1 else max(ld, cols)
    raise ValueError("table must be a 2-D int32 tensor on the current CUDA device with unit inner stride")


def _cache(k_cache, v_cache, dev):
    """Pools (n_pages, n_kv, page_size, head_dim) with unit inner stride and equal strides -> KvCache."""
    shape, st = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or k_cache.get_device() != dev or v_cache.get_device() != dev or st[3] != 1 or shape[3] == 0 or \
            v_cache.shape != shape or v_cache.stride() != st or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must be tensors (n_pages, n_kv, page_size, head_dim) on the current CUDA "
                         "device, of one dtype and equal strides, unit inner stride")
    dtype = _act_types().get(k_cache.dtype)
    if dtype is None or dtype == Q2_0_ACT_F32:
        raise ValueError("the cache must be float16 or bfloat16")
    n_pages, n_kv, page, dim = shape
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), dtype, n_pages, page, n_kv, dim, st[0], st[1], st[2])


def q2_0_kv_append(k_cache, v_cache, table, seq, pos, k, v, rope=None, style: int = Q2_0_ROPE_HALF, q=None, q_out=None,
                   stream=None):
    """Rotate q and k by their positions and store k and v in the paged cache.

    k_cache, v_cache (n_pages, n_kv, page_size, head_dim) float16 or bfloat16, any strides with unit inner
    stride; table (n_seqs, pages) int32 page numbers; seq, pos (n_tokens) int32; k, v (n_tokens, n_kv*head_dim)
    and q (n_tokens, n_q*head_dim) float32, float16 or bfloat16, all of one dtype; rope (n_pos, rot_dim) float32, cos then
    sin of a position's angles (None: no rotation).  Returns the rotated q in the cache's dtype (None without q)."""
    import torch
    dev = torch.cuda.current_device()
    c = _cache(k_cache, v_cache, dev)
    n = k.shape[0] if k.dim() == 2 else -1
    xt = _act_types().get(k.dtype)
    if xt is None or v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise ValueError("q, k and v must be float32, float16 or bfloat16, all of one dtype")
    tp, n_seqs, cols, ldt = _table(table, dev)
    kv = c.n_kv * c.head_dim
    ldk, ldv = _rows(k, n, kv, "k", dev), _rows(v, n, kv, "v", dev)
    qp, ldq, n_q, op, ldo = 0, 0, 0, 0, 0
    if q is not None:
        width = _wide(q, "q")
        n_q = width // c.head_dim
        if width != n_q * c.head_dim:
            raise ValueError("q must have whole heads of %d elements" % c.head_dim)
        ldq, qp = _rows(q, n, width, "q", dev), q.data_ptr()
        if q_out is None:
            q_out = _empty(k_cache, (n, width), k_cache.dtype, stream)
        elif q_out.dtype != k_cache.dtype:
            raise ValueError("q_out must have the cache's dtype")
        ldo, op = _rows(q_out, n, width, "q_out", dev), q_out.data_ptr()
    rp, n_pos, rot = 0, 0, 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.get_device() != dev or rope.dim() != 2 or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous 2-D float32 tensor on the current CUDA device")
        n_pos, rot = rope.shape
        rp = rope.data_ptr()
    _check(kv_append_raw(c, tp, n_seqs, cols, ldt, _dense(seq, torch.int32, (n,), "seq", dev),
                         _dense(pos, torch.int32, (n,), "pos", dev), n, qp, ldq, n_q, k.data_ptr(), ldk, v.data_ptr(), ldv, xt,
                         rp, n_pos, rot, style, op, ldo, _stream(stream, dev)), "q2_0_kv_append")
    return q_out


def q2_0_attn_shared(q, k_cache, v_cache, table, lens, scale: float, prefix_len: int = 0, max_len=None, n_qt: int = 1,
                     out=None, workspace=None, stream=None):
    """Attention of n_qt query tokens per sequence over the paged cache, the first prefix_len tokens shared.

    q (n_seqs*n_qt, n_q*head_dim) of the cache's dtype; table (n_seqs, pages) int32; lens (n_seqs) int32: tokens of
    each sequence with the prefix and its query tokens; max_len bounds lens (default: what the table holds).  Returns
    out like q."""
    import torch
    dev = torch.cuda.current_device()
    c = _cache(k_cache, v_cache, dev)
    tp, n_seqs, cols, ldt = _table(table, dev)
    width = _wide(q, "q")
    n_q = width // c.head_dim
    if q.dtype != k_cache.dtype or width != n_q * c.head_dim:
        raise ValueError("q must have the cache's dtype and whole heads of %d elements" % c.head_dim)
    ldq = _rows(q, n_seqs * n_qt, width, "q", dev)
    if out is None:
        out = _empty(q, (n_seqs * n_qt, width), q.dtype, stream)
    elif out.dtype != q.dtype:
        raise ValueError("out must have the cache's dtype")
    ldo = _rows(out, n_seqs * n_qt, width, "out", dev)
    if max_len is None:
        max_len = cols * c.page_size
    need = attn_shared_workspace_bytes(n_seqs, n_q, c.n_kv, c.head_dim, n_qt, prefix_len, max_len)
    workspace, wsp, wsb = _work(workspace, need, q, stream, dev)
    _check(attn_shared_raw(c, tp, n_seqs, cols, ldt, _dense(lens, torch.int32, (n_seqs,), "lens", dev), prefix_len, max_len,
                           q.data_ptr(), ldq, n_q, n_qt, scale, out.data_ptr(), ldo, wsp, wsb, _stream(stream, dev)),
           "q2_0_attn_shared")
    return out


def q2_0_moe_route(logits, n_used: int, normalise: bool = True, ids=None, weights=None, stream=None):
    """(ids, weights), each (n_tokens, n_used): the n_used largest router logits of each row of logits
    (n_tokens, n_expert) float32, float16 or bfloat16, largest first and the lower index first among equals, and their
    softmax weights over the chosen (normalise) or over all experts."""
    import torch
    dev = torch.cuda.current_device()
    n_expert = _wide(logits, "logits")
    n = logits.shape[0]
    xt = _act_types().get(logits.dtype)
    if xt is None:
        raise ValueError("logits must be float32, float16 or bfloat16")
    ld = _rows(logits, n, n_expert, "logits", dev)
    if ids is None:
        ids = _empty(logits, (n, n_used), torch.int32, stream)
    if weights is None:
        weights = _empty(logits, (n, n_used), torch.float32, stream)
    _check(moe_route_raw(logits.data_ptr(), xt, ld, n, n_expert, n_used, int(bool(normalise)),
                         _dense(ids, torch.int32, (n, n_used), "ids", dev),
                         _dense(weights, torch.float32, (n, n_used), "weights", dev), _stream(stream, dev)), "q2_0_moe_route")
    return ids, weights


def q2_0_moe_layer(w_gate, w_up, w_down, n_expert: int, n_ff: int, K: int, x, ids, weights, y=None, workspace=None,
                   stream=None):
    """y (n_tokens, K) float32 = sum over u of weights[t, u] * W_down (silu(W_gate x) * (W_up x)) of expert ids[t, u].

    w_gate and w_up hold n_expert (n_ff, K) Q2_0 matrices back to back, w_down n_expert (K, n_ff) ones; x (n_tokens, >=K)
    float32, float16 or bfloat16, at most MOE_LAYER_MAX_TOKENS rows; ids int32 and weights float32 (n_tokens, n_used)."""
    import torch
    dev = torch.cuda.current_device()
    xp, n, ldx, xt = _xcols(x, K, "x")
    n_used = _wide(ids, "ids")
    for w, name in ((w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        if w.get_device() != dev or not w.is_contiguous() or \
                w.numel() * w.element_size() < n_expert * n_ff * K // BLOCK_WEIGHTS * BLOCK_BYTES:
            raise ValueError("%s must be a contiguous tensor on the current CUDA device that holds n_expert matrices" % name)
    if y is None:
        y = _empty(x, (n, K), torch.float32, stream)
    yp, yn, ldy = _cols(y, K, "y")
    if yn != n:
        raise ValueError("y must have n_tokens rows")
    if x.get_device() != dev or y.get_device() != dev:
        raise ValueError("x and y must be on the current CUDA device")
    need = moe_layer_workspace_bytes(n_ff, K, n_used, n)
    workspace, wsp, wsb = _work(workspace, need, x, stream, dev)
    _check(moe_layer_raw(w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), n_expert, n_ff, K, xp, xt, ldx,
                         _dense(ids, torch.int32, (n, n_used), "ids", dev),
                         _dense(weights, torch.float32, (n, n_used), "weights", dev), n_used, n, yp, ldy, wsp, wsb,
                         _stream(stream, dev)), "q2_0_moe_layer")
    return y


# ------------------------------------------------------------- between two decoder steps (torch)

def _ints(t, name, dev):
    """A contiguous 1-D int32 tensor -> (address, length)."""
    import torch
    if t.dtype != torch.int32 or t.get_device() != dev or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous 1-D int32 tensor on the current CUDA device" % name)
    return t.data_ptr(), t.shape[0]


def _result(t, like, shape, dtype, name, stream, dev):
    """A result given, or a new one -> (tensor, address)."""
    if t is None:
        t = _empty(like, shape, dtype, stream)
        return t, t.data_ptr()
    return t, _dense(t, dtype, shape, name, dev)


def _pages(ref, free, n_pages, dev):
    """Counts and free bits (int32, 32 pages a word) of n_pages pages -> KvPages."""
    import torch
    return KvPages(_dense(ref, torch.int32, (n_pages,), "ref", dev),
                   _dense(free, torch.int32, ((n_pages + 31) // 32,), "free", dev), n_pages)


def q2_0_kv_pages(n_pages: int, device="cuda"):
    """(ref, free) of a new pool of n_pages pages, all free: int32 counts, and int32 words of 32 pages' bits."""
    import torch
    return torch.zeros(n_pages, dtype=torch.int32, device=device), \
        torch.full(((n_pages + 31) // 32,), -1, dtype=torch.int32, device=device)


def q2_0_moe_route_groups(logits, n_used: int, score: int = Q2_0_SCORE_SIGMOID, bias=None, n_group: int = 1,
                          n_group_used: int = 1, group_top: int = 1, normalise: bool = True, scale: float = 1.0, ids=None,
                          weights=None, stream=None):
    """(ids, weights), each (n_tokens, n_used): the n_used experts of the largest score + bias in the n_group_used best of
    n_group groups (by the sum of a group's group_top largest), largest first and the lower index first among equals, and
    scale * score, over the chosen scores' sum with normalise.  logits (n_tokens, n_expert) float32, float16 or bfloat16;
    score Q2_0_SCORE_SIGMOID or Q2_0_SCORE_SOFTMAX; bias (n_expert) float32 or None, for the choice alone."""
    import torch
    dev = torch.cuda.current_device()
    n_expert = _wide(logits, "logits")
    n = logits.shape[0]
    xt = _act_types().get(logits.dtype)
    if xt is None:
        raise ValueError("logits must be float32, float16 or bfloat16")
    ld = _rows(logits, n, n_expert, "logits", dev)
    bp = 0 if bias is None else _dense(bias, torch.float32, (n_expert,), "bias", dev)
    ids, ip = _result(ids, logits, (n, n_used), torch.int32, "ids", stream, dev)
    weights, wp = _result(weights, logits, (n, n_used), torch.float32, "weights", stream, dev)
    _check(moe_route_groups_raw(logits.data_ptr(), xt, ld, n, n_expert, n_used, score, bp, n_group, n_group_used, group_top,
                                int(bool(normalise)), scale, ip, wp, _stream(stream, dev)), "q2_0_moe_route_groups")
    return ids, weights


def q2_0_draft_verify(target, draft, tokens, n_draft, u, form: int = Q2_0_DRAFT_LOGITS, temperature=None, out=None,
                      n_accepted=None, workspace=None, stream=None):
    """(out (n_seqs, max_draft + 1), n_accepted (n_seqs)), int32: the drafted tokens that the target takes, the token that
    follows them, then -1; and how many are taken.

    target (n_seqs*(max_draft+1), n_vocab) and draft (n_seqs*max_draft, n_vocab; None: drafts that were found, not drawn)
    float32, float16 or bfloat16, both logits or both probabilities (form); tokens (n_seqs, max_draft) and n_draft (n_seqs)
    int32; u (n_seqs, max_draft + 1) float32 of [0, 1); temperature (n_seqs) float32, 0 for the largest logit."""
    import torch
    dev = torch.cuda.current_device()
    n, most = n_draft.shape[0] if n_draft.dim() == 1 else -1, _wide(tokens, "tokens")
    vocab = _wide(target, "target")
    xt = _act_types().get(target.dtype)
    if xt is None or (draft is not None and draft.dtype != target.dtype):
        raise ValueError("target and draft must be float32, float16 or bfloat16, both of one dtype")
    ldt = _rows(target, n * (most + 1), vocab, "target", dev)
    dp, ldd = 0, 0
    if draft is not None:
        if _wide(draft, "draft") != vocab:
            raise ValueError("draft must have as many columns as target")
        dp, ldd = draft.data_ptr(), _rows(draft, n * most, vocab, "draft", dev)
    tp = 0 if temperature is None else _dense(temperature, torch.float32, (n,), "temperature", dev)
    out, op = _result(out, target, (n, most + 1), torch.int32, "out", stream, dev)
    n_accepted, ap = _result(n_accepted, target, (n,), torch.int32, "n_accepted", stream, dev)
    need = draft_verify_workspace_bytes(n, most, vocab, xt, form, int(draft is not None))
    workspace, wsp, wsb = _work(workspace, need, target, stream, dev)
    _check(draft_verify_raw(target.data_ptr(), ldt, dp, ldd, xt, form, vocab, tp,
                            _dense(tokens, torch.int32, (n, most), "tokens", dev),
                            _dense(n_draft, torch.int32, (n,), "n_draft", dev),
                            _dense(u, torch.float32, (n, most + 1), "u", dev), n, most, op, ap, wsp, wsb, _stream(stream, dev)),
           "q2_0_draft_verify")
    return out, n_accepted


def q2_0_kv_copy(k_to, v_to, k_from, v_from, src, dst, stream=None):
    """Copies pages src[i] of the pools k_from, v_from to pages dst[i] of k_to, v_to (the same pools, or others of the same
    page): src, dst int32, pairs outside the pools are left out."""
    import torch
    dev = torch.cuda.current_device()
    to, frm = _cache(k_to, v_to, dev), _cache(k_from, v_from, dev)
    sp, n = _ints(src, "src", dev)
    _check(kv_copy_raw(to, frm, sp, _dense(dst, torch.int32, (n,), "dst", dev), n, _stream(stream, dev)), "q2_0_kv_copy")


def q2_0_kv_fork(ref, table, page_size: int, lens, src, dst, workspace=None, stream=None):
    """Sequence dst[i] (empty) becomes one of the same tokens as src[i], in the same pages: table, lens and ref change.

    ref (n_pages), lens (n_seqs), src and dst (n) int32; table (n_seqs, pages) int32."""
    import torch
    dev = torch.cuda.current_device()
    tp, n_seqs, cols, ldt = _table(table, dev)
    rp, n_pages = _ints(ref, "ref", dev)
    sp, n = _ints(src, "src", dev)
    workspace, wsp, wsb = _work(workspace, kv_fork_workspace_bytes(n), ref, stream, dev)
    _check(kv_fork_raw(rp, n_pages, tp, n_seqs, cols, ldt, page_size, _dense(lens, torch.int32, (n_seqs,), "lens", dev), sp,
                       _dense(dst, torch.int32, (n,), "dst", dev), n, wsp, wsb, _stream(stream, dev)), "q2_0_kv_fork")


def q2_0_kv_resize(k_cache, v_cache, ref, free, table, lens, new_lens, missing=None, workspace=None, stream=None):
    """Every sequence gets the length new_lens[s] (-1: as it is): the pages that it leaves go back, those that it needs are
    taken, and a shared page that it would write in becomes a copy of its own.  table, lens, ref, free and the pools change.
    Returns missing (1) int32: 0, or how many free pages too few there are (then no sequence has grown).

    ref (n_pages) and free ((n_pages + 31) // 32) as q2_0_kv_pages gives them; table (n_seqs, pages), lens and new_lens
    (n_seqs) int32."""
    import torch
    dev = torch.cuda.current_device()
    c = _cache(k_cache, v_cache, dev)
    tp, n_seqs, cols, ldt = _table(table, dev)
    missing, mp = _result(missing, lens, (1,), torch.int32, "missing", stream, dev)
    if n_seqs == 0:                       # (the library writes nothing then)
        _stream(stream, dev)
        other = None if stream is None else _other(stream)
        with torch.cuda.stream(other) if other is not None else contextlib.nullcontext():
            return missing.zero_()
    workspace, wsp, wsb = _work(workspace, kv_resize_workspace_bytes(n_seqs, c.n_pages), lens, stream, dev)
    _check(kv_resize_raw(c, _pages(ref, free, c.n_pages, dev), tp, n_seqs, cols, ldt,
                         _dense(lens, torch.int32, (n_seqs,), "lens", dev),
                         _dense(new_lens, torch.int32, (n_seqs,), "new_lens", dev), mp, wsp, wsb, _stream(stream, dev)),
           "q2_0_kv_resize")
    return missing


def q2_0_kv_compact(k_to, v_to, ref_to, free_to, table_to, k_from, v_from, ref, free, table, lens, n_used=None,
                    workspace=None, stream=None):
    """Moves the pages that are not free from the pools k_from, v_from to the first pages of k_to, v_to, in order, and writes
    their counts, bits and table rows there.  Returns n_used (1) int32: how many there are; more than the new pools
    hold: nothing else is written.  table_to like table (n_seqs, pages) int32; lens (n_seqs) int32."""
    import torch
    dev = torch.cuda.current_device()
    to, frm = _cache(k_to, v_to, dev), _cache(k_from, v_from, dev)
    tp, n_seqs, cols, ldt = _table(table, dev)
    np_, n_to, cols_to, ldn = _table(table_to, dev)
    if n_to != n_seqs or cols_to != cols:
        raise ValueError("table_to must have the shape of table")
    n_used, up = _result(n_used, lens, (1,), torch.int32, "n_used", stream, dev)
    workspace, wsp, wsb = _work(workspace, kv_compact_workspace_bytes(frm.n_pages), lens, stream, dev)
    _check(kv_compact_raw(to, _pages(ref_to, free_to, to.n_pages, dev), frm, _pages(ref, free, frm.n_pages, dev), tp, n_seqs,
                          cols, ldt, _dense(lens, torch.int32, (n_seqs,), "lens", dev), np_, ldn, up, wsp, wsb,
                          _stream(stream, dev)), "q2_0_kv_compact")
    return n_used
