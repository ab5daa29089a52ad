// Position rotation of q and k and the store of k and v into a paged cache, one launch.
//
// A pair (a, b) of a head's first rot elements becomes (a c - b s, b c + a s) with c, s =
// cos, sin of the token's position from the caller's table, in f32, rounded once to the
// cache's type; v and the elements past rot are only rounded.
//
// Work: a thread takes 8 elements of one head (kv_append_vec): with rot/2 a multiple of 4 a
// unit is either 4 pairs -- 4 + 4 elements half a rotation apart, or 8 in a row for adjacent
// pairs -- which need the same 4 cosines and sines in both styles, or 8 elements past the
// rotation.  Loads and stores are 8 or 16 bytes wide and neighbouring threads touch
// neighbouring addresses.  kv_append_any does one pair per thread for everything the vector
// form does not take: unaligned rows, rot/2 not a multiple of 4.
//
// What bounds it: a launch and three dependent loads (position, page, row) for one token (32 + 8 + 8 heads
// of 128: 2.6 us in a graph), HBM for many: 4099 tokens of f32 into a bfloat16 cache, 101 MB read and
// 50 MB written, 24.9 us, 6.1 TB/s, where a copy of 2 GiB runs at 5.0.
#include "q2_0_internal.h"
#include "layer_common.h"

namespace q2_0 {

// A token's destination row in the cache, in elements without the head term; < 0: none.
__device__ __forceinline__ int64_t cache_row(const KvAppend &a, int seq, int pos) {
    if (seq < 0 || seq >= a.n_seqs || pos < 0) return -1;
    const int pi = a.page.div((uint32_t)pos);
    if (pi >= a.table_len) return -1;
    const int page = a.table[(int64_t)seq * a.ld_table + pi];
    if (page < 0 || page >= a.n_pages) return -1;
    return (int64_t)page * a.page_stride + (int64_t)(pos - pi * (int)a.page.d) * a.token_stride;
}

template <typename XT>
__device__ __forceinline__ float4_t load_src4(const XT *p) {
    return load_act4(p);
}

template <typename CT>
__device__ __forceinline__ void store4(CT *p, float4_t v) {
    *reinterpret_cast<u32x2_t *>(p) = u32x2_t{pack2<CT>(v.x, v.y), pack2<CT>(v.z, v.w)};
}

template <typename CT>
__device__ __forceinline__ void store8(CT *p, float4_t u, float4_t v) {
    *reinterpret_cast<u32x4_t *>(p) =
        u32x4_t{pack2<CT>(u.x, u.y), pack2<CT>(u.z, u.w), pack2<CT>(v.x, v.y), pack2<CT>(v.z, v.w)};
}

// Source row, destination row and kind of head hd (q heads, then k, then v) of token t;
// returns false where there is nothing to write.
template <typename XT, typename CT>
__device__ __forceinline__ bool head_rows(const KvAppend &a, int64_t t, int hd, const XT *&src, CT *&dst, bool &turn) {
    if (hd < a.n_q) {
        src = static_cast<const XT *>(a.q) + t * a.ldq + (int64_t)hd * a.dim;
        dst = static_cast<CT *>(a.q_out) + t * a.ldqo + (int64_t)hd * a.dim;
        turn = true;
        return true;
    }
    const int64_t row = cache_row(a, a.seq[t], a.pos[t]);
    if (row < 0) return false;
    const bool is_k = hd < a.n_q + a.n_kv;
    const int h = hd - a.n_q - (is_k ? 0 : a.n_kv);
    src = static_cast<const XT *>(is_k ? a.k : a.v) + t * (is_k ? a.ldk : a.ldv) + (int64_t)h * a.dim;
    dst = static_cast<CT *>(is_k ? a.kc : a.vc) + row + (int64_t)h * a.head_stride;
    turn = is_k;
    return true;
}

template <typename XT, typename CT, bool HALF>
__global__ __launch_bounds__(256) void kv_append_vec(KvAppend a) {
    const int upd = a.dim / 8;                         // units per head: 8, 16 or 32
    const int unit = threadIdx.x & (upd - 1);
    const int64_t t = blockIdx.x / (unsigned)a.head_blocks;
    const int hd = (int)(blockIdx.x % (unsigned)a.head_blocks) * (256 / upd) + (int)(threadIdx.x / (unsigned)upd);
    if (hd >= a.n_q + 2 * a.n_kv) return;
    const XT *src;
    CT *dst;
    bool turn;
    if (!head_rows<XT, CT>(a, t, hd, src, dst, turn)) return;
    const int half = a.rot / 2;
    if (!turn || 8 * unit >= a.rot) {
        store8(dst + 8 * unit, load_src4(src + 8 * unit), load_src4(src + 8 * unit + 4));
        return;
    }
    const int i0 = HALF ? 4 * unit : 8 * unit, i1 = HALF ? half + 4 * unit : 8 * unit + 4;
    const float4_t u = load_src4(src + i0), w = load_src4(src + i1);
    const int pos = a.pos[t];
    float4_t c, s;
    if (pos >= 0 && pos < a.n_pos) {
        const float *r = a.rope + (int64_t)pos * a.rot + 4 * unit;
        c = *reinterpret_cast<const float4_t *>(r);
        s = *reinterpret_cast<const float4_t *>(r + half);
    } else {
        c = s = float4_t{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    }
    if (HALF) {
        float4_t x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = u[i] * c[i] - w[i] * s[i];
            y[i] = w[i] * c[i] + u[i] * s[i];
        }
        store4(dst + i0, x);
        store4(dst + i1, y);
    } else {
        const float a0[4] = {u.x, u.z, w.x, w.z}, b0[4] = {u.y, u.w, w.y, w.w};
        float o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = a0[i] * c[i] - b0[i] * s[i];
            o[2 * i + 1] = b0[i] * c[i] + a0[i] * s[i];
        }
        store8(dst + i0, float4_t{o[0], o[1], o[2], o[3]}, float4_t{o[4], o[5], o[6], o[7]});
    }
}

template <typename XT, typename CT>
__global__ __launch_bounds__(256) void kv_append_any(KvAppend a) {
    const int ppd = a.dim / 2;                         // pairs per head: 32, 64 or 128
    const int i = threadIdx.x & (ppd - 1);
    const int64_t t = blockIdx.x / (unsigned)a.head_blocks;
    const int hd = (int)(blockIdx.x % (unsigned)a.head_blocks) * (256 / ppd) + (int)(threadIdx.x / (unsigned)ppd);
    if (hd >= a.n_q + 2 * a.n_kv) return;
    const XT *src;
    CT *dst;
    bool turn;
    if (!head_rows<XT, CT>(a, t, hd, src, dst, turn)) return;
    const int half = a.rot / 2;
    const bool in = i < half;
    const int ia = in && a.half_style ? i : 2 * i;     // pairs past the rotation: adjacent elements
    const int ib = in && a.half_style ? i + half : 2 * i + 1;
    float x = act_to_f32(src[ia]), y = act_to_f32(src[ib]);
    if (turn && in) {
        const int pos = a.pos[t];
        float c = __builtin_nanf(""), s = c;
        if (pos >= 0 && pos < a.n_pos) {
            c = a.rope[(int64_t)pos * a.rot + i];
            s = a.rope[(int64_t)pos * a.rot + half + i];
        }
        const float r = x * c - y * s;
        y = y * c + x * s;
        x = r;
    }
    dst[ia] = to_elem<CT>(x);
    dst[ib] = to_elem<CT>(y);
}

static bool vector_form(const KvAppend &a, Act xt) {
    const int eb = act_bytes(xt);
    const auto fits = [&](const void *p, int64_t ld) { return (uintptr_t)p % (4 * eb) == 0 && ld % 4 == 0; };
    return a.rot % 8 == 0 && (a.n_q == 0 || (fits(a.q, a.ldq) && (uintptr_t)a.q_out % 16 == 0 && a.ldqo % 8 == 0)) &&
           fits(a.k, a.ldk) && fits(a.v, a.ldv) && (uintptr_t)a.rope % 16 == 0;
}

static int head_blocks(const KvAppend &a, bool vec) {
    const int per = vec ? 256 / (a.dim / 8) : 256 / (a.dim / 2);    // heads per workgroup
    return (a.n_q + 2 * a.n_kv + per - 1) / per;
}

int64_t kv_append_groups(const KvAppend &a, Act xt, int64_t n_tokens) {
    return n_tokens * head_blocks(a, vector_form(a, xt));
}

hipError_t launch_kv_append(KvAppend a, Act xt, Act ct, int64_t n_tokens, hipStream_t s) {
    const bool vec = vector_form(a, xt);
    a.head_blocks = head_blocks(a, vec);
    const dim3 grid((unsigned)(n_tokens * a.head_blocks));
    return with_act(xt, [&](auto xtag) -> hipError_t {
        using XT = decltype(xtag);
        auto go = [&](auto ctag) {
            using CT = decltype(ctag);
            if (!vec) kv_append_any<XT, CT><<<grid, 256, 0, s>>>(a);
            else if (a.half_style) kv_append_vec<XT, CT, true><<<grid, 256, 0, s>>>(a);
            else kv_append_vec<XT, CT, false><<<grid, 256, 0, s>>>(a);
        };
        if (ct == Act::F16) go(_Float16{});
        else go(bf16_t{});
        return hipGetLastError();
    });
}

}  // namespace q2_0
