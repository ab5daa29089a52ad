// Shared by the decoder-step operators (cache append, attention, expert choice and layer).
#pragma once

#include "q2_0_internal.h"

namespace q2_0 {

// n / d for 0 <= n < 2^31 and a divisor fixed at the launch, as a multiply-high: with
// s = ceil(log2 d) and m = ceil(2^(31+s) / d) the error n * (m d - 2^(31+s)) / (d 2^(31+s)) stays
// under 1/d, and m fits 32 bits.
struct FastDiv {
    uint32_t d, m, s;
    static FastDiv make(uint32_t d) {
        uint32_t s = 0;
        while (((uint64_t)1 << s) < d) ++s;
        const uint64_t p = (uint64_t)1 << (31 + s);
        return FastDiv{d, (uint32_t)((p + d - 1) / d), s};
    }
    __device__ __forceinline__ int div(uint32_t n) const {
        return (int)(((uint64_t)n * m) >> (31 + s));
    }
};

// f32 -> one element of a 16-bit type, nearest, ties to even
template <typename CT>
__device__ __forceinline__ CT to_elem(float v);
template <>
__device__ __forceinline__ _Float16 to_elem<_Float16>(float v) { return (_Float16)v; }
template <>
__device__ __forceinline__ bf16_t to_elem<bf16_t>(float v) { return __builtin_bit_cast(bf16_t, (__bf16)v); }

// two of them packed, a in the low half
template <typename CT>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<_Float16>(float a, float b) {
    return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
}
template <>
__device__ __forceinline__ uint32_t pack2<bf16_t>(float a, float b) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf2{(__bf16)a, (__bf16)b});
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
    return v > o ? v : o;
}

// Maximum over the wave, uniform: row shifts by 1, 2, 4, 8, then the row broadcasts.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = dpp_max<0x111>(v);
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142>(v);
    v = dpp_max<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

struct KvAppend {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    void *q_out;
    int64_t ldqo;
    void *kc, *vc;
    int64_t page_stride, head_stride, token_stride;
    const int32_t *table;
    int64_t ld_table, n_seqs, table_len, n_pages;
    const int32_t *seq, *pos;
    const float *rope;
    int64_t n_pos;
    FastDiv page;
    int n_q, n_kv, dim, rot, half_style;
    int head_blocks;      // workgroups per token
};
int64_t kv_append_groups(const KvAppend &a, Act xt, int64_t n_tokens);   // workgroups of the launch
hipError_t launch_kv_append(KvAppend a, Act xt, Act ct, int64_t n_tokens, hipStream_t s);

hipError_t launch_moe_choose(const void *logits, Act xt, int64_t ld, int64_t n_tokens, int n_expert, int n_used,
                             int normalise, int32_t *ids, float *weights, hipStream_t s);

// ---- attention over a shared prefix and the sequences' own keys
struct AttnShared {
    const void *q;
    int64_t ldq;
    const void *kc, *vc;
    int64_t page_stride, head_stride, token_stride;
    const int32_t *table;
    int64_t ld_table, n_pages;
    const int32_t *lens;
    void *out;
    int64_t ldo;
    float *part_o;        // [row][split][dim], row = query row * n_q + head
    float *part_ml;       // [row][split][2]: reference exponent, sum
    FastDiv page, group, heads, queries;   // tokens per page, query heads per key head, key heads, query tokens
    float scale2;         // scale * log2(e)
    int n_seqs, n_qt, n_q, n_kv;
    int prefix_len, max_len;
    // the launch: prefix workgroups first, then own ones
    int rows_p, splits_p, wgs_p;           // rows of a key head, splits and workgroups of the prefix
    int rows_o, wgs_o;                     // the same for one sequence's own keys
    FastDiv groups_p, groups_o, splits_o, div_p;   // row groups; splits
    int own_from, joint_len;               // first key of the own part; its keys below this are the prefix's (row 0)
    int xcd_p;                             // row groups of the same prefix keys 8 workgroups apart
};
struct AttnPlan {
    int row_tiles;                         // 16-row tiles of a wave in the prefix part; 0: no such part
    bool joint;                            // the own part takes the prefix too
    int64_t groups_p, splits_p, groups_o, splits_o;
    int64_t groups;                        // workgroups of the larger launch
    size_t ws_bytes;
};
AttnPlan attn_plan(int64_t n_seqs, int64_t n_q, int64_t n_kv, int64_t dim, int64_t n_qt, int64_t prefix_len,
                   int64_t max_len);
hipError_t launch_attn_shared(AttnShared a, const AttnPlan &p, Act ct, int dim, hipStream_t s);

// ---- expert layer
size_t moe_layer_ws_bytes(int64_t n_ff, int64_t K, int64_t n_used, int64_t n_tokens);
hipError_t launch_moe_layer(const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, int n_expert, int n_ff, int K,
                            const void *x, Act xt, int64_t ldx, const int32_t *ids, const float *weights, int n_used,
                            int n_tokens, float *y, int64_t ldy, void *ws, hipStream_t s);

}  // namespace q2_0
