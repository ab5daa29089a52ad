// Shared by the operators between two decoder steps: grouped expert choice, verification of
// drafted tokens, pages of the cache.
#pragma once

#include "layer_common.h"

namespace q2_0 {

// ---- launches
// One launch and its own status: what another call left as the last error is neither taken for this one's (the rest of a
// call would not run) nor cleared.
template <typename... A, typename... B>
inline hipError_t launch(void (*kernel)(A...), unsigned groups, unsigned threads, size_t lds, hipStream_t s, B... args) {
    return [&](A... exact) {
        void *at[] = {&exact...};
        return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3(groups), dim3(threads), at, lds, s);
    }(args...);
}

// ---- lanes
// A lane's value (`none` where there is no such lane or the row of 16 is not of ROWS) by the lane moves that need no LDS: CTRL 0x111 ..
// 0x118 from 1 .. 8 lanes below in the row, 0x142 and 0x143 the last of the row, and of the rows, before.
template <int CTRL, int ROWS>
__device__ __forceinline__ float lane_move(float v, float none) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), CTRL, ROWS,
                                                                 0xf, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double lane_move(double v) {
    const u32x2_t b = __builtin_bit_cast(u32x2_t, v);
    const uint32_t lo = b.x, hi = b.y;
    const u32x2_t o = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)lo, CTRL, ROWS, 0xf, false),
                       (uint32_t)__builtin_amdgcn_update_dpp(0, (int)hi, CTRL, ROWS, 0xf, false)};
    return __builtin_bit_cast(double, o);
}
// Sums over the lanes up to each, in a fixed order; all 64 lanes.
__device__ __forceinline__ double lanes_run(double v) {
    v += lane_move<0x111, 0xf>(v);
    v += lane_move<0x112, 0xf>(v);
    v += lane_move<0x114, 0xf>(v);
    v += lane_move<0x118, 0xf>(v);
    v += lane_move<0x142, 0xa>(v);
    v += lane_move<0x143, 0xc>(v);
    return v;
}
__device__ __forceinline__ double last_lane(double v) {
    const u32x2_t b = __builtin_bit_cast(u32x2_t, v);
    const uint32_t lo = b.x, hi = b.y;
    const u32x2_t o = {(uint32_t)__builtin_amdgcn_readlane((int)lo, 63), (uint32_t)__builtin_amdgcn_readlane((int)hi, 63)};
    return __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double wave_sum(double v) { return last_lane(lanes_run(v)); }
template <int CTRL, int ROWS>
__device__ __forceinline__ int lane_move(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int lanes_run(int v) {
    v += lane_move<0x111, 0xf>(v);
    v += lane_move<0x112, 0xf>(v);
    v += lane_move<0x114, 0xf>(v);
    v += lane_move<0x118, 0xf>(v);
    v += lane_move<0x142, 0xa>(v);
    v += lane_move<0x143, 0xc>(v);
    return v;
}

// ---- expert choice in groups
struct ChooseGroups {
    const void *logits;
    int64_t ld, n_tokens;
    const float *bias;
    FastDiv size;          // experts of a group
    int n_expert, n_used, n_group, n_group_used, group_top;
    int group_lanes;       // lanes whose keys are a group, a power of two (0: no groups, or of another size)
    int normalise;
    float scale;
    int32_t *ids;
    float *weights;
};
hipError_t launch_moe_choose_groups(ChooseGroups a, Act xt, bool sigmoid, hipStream_t s);

// ---- verification of drafted tokens
struct DraftPlan {
    int64_t stat_groups;   // workgroups of the statistics (0: probabilities are given)
    int64_t sum_groups;    // of the tile sums, sum_parts of a sequence
    int sum_parts;
    int chunks;            // of a row in the statistics
    int chunk_vecs;        // 16-byte vectors of a chunk
    int tiles;             // of a row in the tile sums
    size_t off_z, off_max, off_arg, off_tiles, off_done, off_pick;
    size_t ws_bytes;
};
struct DraftVerify {
    const void *target, *draft;
    int64_t ld_target, ld_draft;
    int n_vocab, n_seqs, max_draft;
    const float *temperature;
    const int32_t *tokens, *n_draft;
    const float *u;
    int32_t *out, *n_accepted;
    char *ws;
};
DraftPlan draft_plan(int64_t n_seqs, int64_t max_draft, int64_t n_vocab, bool has_draft, int elem_bytes, bool probs);
hipError_t launch_draft_verify(const DraftVerify &a, const DraftPlan &p, Act xt, bool probs, hipStream_t s);

// ---- pages of a cache
struct PageRows {          // where the rows of a page are in the two pools
    char *k, *v;
    int64_t page_stride, head_stride, token_stride;   // bytes
};
struct PageShape {
    FastDiv page;          // token rows of a page
    int heads;             // key heads
    int vec_shift;         // log2 of the 16-byte vectors of a row
    int vecs;              // of a page: both pools, all heads and rows
};
struct PageTable {
    int32_t *table;
    int64_t ld;
    int n_seqs, cols;
    int32_t *lens;
};
struct KvCopy {
    PageRows to, from;
    PageShape shape;
    int to_pages, from_pages;
    const int32_t *src, *dst;
    int n;
};
hipError_t launch_kv_copy(const KvCopy &a, hipStream_t s);
int64_t kv_copy_groups(const PageShape &p, int64_t n);

struct KvFork {
    PageTable t;
    FastDiv page;
    int32_t *ref;
    int n_pages, n;
    const int32_t *src, *dst;
    int32_t *plan;         // length that pair i copies, -1: none
};
hipError_t launch_kv_fork(const KvFork &a, hipStream_t s);
int64_t kv_table_groups(int64_t n_rows, int64_t cols);

constexpr int kResizeMaxSeqs = 8192;
struct KvResize {
    PageTable t;
    PageRows rows;
    PageShape shape;
    int32_t *ref;
    uint32_t *free;
    int n_pages;
    const int32_t *new_lens;
    int32_t *missing;
    int32_t *plan;         // 8 numbers a sequence
    int32_t *fresh;        // the pages that the call takes
    int32_t *before;       // free pages before each word of `free` (large tables), how many are taken, and of how many words
};
hipError_t launch_kv_resize(const KvResize &a, hipStream_t s);

struct KvCompact {
    PageTable t;
    PageRows to, from;
    PageShape shape;
    const int32_t *ref;
    const uint32_t *free;
    int from_pages, to_pages;
    int32_t *to_ref;
    uint32_t *to_free;
    int32_t *to_table;
    int64_t ld_to;
    int32_t *n_used;
    int32_t *before;       // pages in use before each word of `free`
};
hipError_t launch_kv_compact(const KvCompact &a, hipStream_t s);

}  // namespace q2_0
