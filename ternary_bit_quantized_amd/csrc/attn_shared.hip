// Attention of a batch over a paged cache, the prefix that the sequences share read once.
//
//   o[r] = sum_i p_ri v_i / sum_i p_ri,   p_ri = 2^(c q_r.k_i - m_r),   c = scale log2 e
//
// The softmax is one pass: a wave keeps a reference exponent m_r, the sum l_r and the
// unnormalised O_r (f32) of its rows; two results over different keys join as
// l = l1 2^(m1-m) + l2 2^(m2-m), O likewise, with m = max(m1, m2).
//
// Rows.  A key head's rows are (query token, query head of its group).  In the prefix part
// the rows of all sequences stand together (the keys are read once for all of them), in the
// own part those of one sequence.  A wave carries RT tiles of 16 rows.
//
// Keys.  A wave takes 32 keys at a time straight from the cache into the matrix cores'
// operands, without LDS:
//  * S^T = K Q^T (v_mfma 16x16x32): A = 16 keys x 32 dims, 16 bytes a lane, as they lie in
//    the cache; B = Q^T, loaded once.  D: lane (row j = lane%16, g = lane/16) holds the
//    scores of keys 4g..4g+3 of each 16-key half for row j.
//  * O^T += V^T P^T: B = P^T needs, in lane (j, g), 8 keys of row j: exactly the two
//    halves' scores of that lane, rounded.  A = V^T takes the same 8 keys {4g+i, 16+4g+i} of
//    dims d = DPL*c + e (c = lane%16, one MFMA per e): a lane loads DPL consecutive dims
//    of those 8 value rows (full rows across the 16 lanes) and pairs keys up with one
//    v_perm_b32 a dword.
// So a score never leaves its lane: no lane exchange per step.  The reference m_r is only
// raised when some score passes it by 2^8 (a ballot decides), and the sum of a row stays
// spread over its four lanes until the end; f32 has room for terms up to 2^8 and the 16-bit
// P for them too.
//
// Masks.  A row sees keys below its limit.  Scores past it become -inf before the maximum, value
// rows nobody sees are zeroed, and tiles whose keys only some of the wave's rows see (draft tokens,
// sequences shorter than the prefix) go through a loop of their own, so that what lies in
// unseen places (NaN, inf) reaches no row that does not see it.  Addresses are clamped to seen keys.
//
// Split.  The waves of a workgroup interleave the key tiles of one split; their results join in
// LDS, the splits' in attn_join.  Workgroups that read the same prefix keys for other rows get
// launch numbers 8 apart: the same XCD, whose L2 then serves all but one of them.
#include <type_traits>

#include "layer_common.h"

namespace q2_0 {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

template <typename CT>
struct Mma;
template <>
struct Mma<_Float16> {
    static __device__ __forceinline__ float4_t mul(u32x4_t a, u32x4_t b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c,
                                                      0, 0, 0);
    }
};
template <>
struct Mma<bf16_t> {
    static __device__ __forceinline__ float4_t mul(u32x4_t a, u32x4_t b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, a), __builtin_bit_cast(bf8_t, b), c, 0,
                                                       0, 0);
    }
};

// Past every wait state of the matrix instructions before it.  The compiler inserts those that a read
// of their results needs within a block, but was seen to leave them out at a branch's target
// (results then came out wrong now and then); so one stands before such branches.
__device__ __forceinline__ void settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15");
    __builtin_amdgcn_sched_barrier(0);
}

constexpr int kAttnTile = 32;    // keys per step
constexpr int kAttnMaxSplits = 32;

template <int CTRL>
__device__ __forceinline__ int dpp_int(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}

// Over the 16 lanes of a DPP row (row_ror 8, 4, 2, 1).
__device__ __forceinline__ int row_min(int v) {
    v = min(v, dpp_int<0x128>(v));
    v = min(v, dpp_int<0x124>(v));
    v = min(v, dpp_int<0x122>(v));
    return min(v, dpp_int<0x121>(v));
}

// N dwords from 4-byte aligned memory (8 or 16 bytes aligned as N goes)
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t *p, uint32_t *v) {
    if constexpr (N == 2) {
        const u32x2_t t = *reinterpret_cast<const u32x2_t *>(p);
        v[0] = t.x, v[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4_t t = *reinterpret_cast<const u32x4_t *>(p + 4 * i);
            v[i] = t.x, v[i + 1] = t.y, v[i + 2] = t.z, v[i + 3] = t.w;
        }
    }
}

// W: waves.  P16: page_size % 16 == 0 (and the keys start at a multiple of 16, or are all of one page
// table row), so that the 16 keys of a half tile lie in one page and its page number is read
// once for the wave; otherwise 32 lanes look up a key each and pass the rows round through LDS.
template <typename CT, int D, int RT, int W, bool P16>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attn_rows(AttnShared a) {
    constexpr int KS = D / 32;       // 32-dim steps of a score
    constexpr int DPL = D / 16;      // dims per lane of a value row
    constexpr int VD = DPL / 2;      // dwords of those
    constexpr int OS = D + 4;        // LDS floats per row

    __shared__ __attribute__((aligned(16))) float lds_o[W][RT * 16][OS];
    __shared__ float lds_m[W][RT * 16], lds_l[W][RT * 16];
    __shared__ int64_t lds_row[P16 ? 1 : W][P16 ? 1 : kAttnTile];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g = lane >> 4;

    // this workgroup's part: prefix (all sequences' rows) or one sequence's own keys
    const bool pre = (int)blockIdx.x < a.wgs_p;
    const int nrows = pre ? a.rows_p : a.rows_o;
    int rg, kvh, split, seq = 0;
    if (pre) {
        const int id = blockIdx.x, x = a.xcd_p ? id & 7 : 0, y = a.xcd_p ? id >> 3 : id;
        int u = a.groups_p.div((uint32_t)y);
        rg = y - u * (int)a.groups_p.d;
        if (a.xcd_p) u = u * 8 + x;
        split = a.heads.div((uint32_t)u);
        kvh = u - split * a.n_kv;
    } else {
        const int id = (int)blockIdx.x - a.wgs_p;
        int u = a.groups_o.div((uint32_t)id);
        rg = id - u * (int)a.groups_o.d;
        int v = a.heads.div((uint32_t)u);
        kvh = u - v * a.n_kv;
        seq = a.splits_o.div((uint32_t)v);
        split = v - seq * (int)a.splits_o.d;
    }
    const int splits = pre ? a.splits_p : (int)a.splits_o.d;
    const int r0 = rg * RT * 16;
    const int tok0 = seq * a.n_qt;

    // a row's query (token, head) and the keys it sees
    const int grp = (int)a.group.d;
    const auto row_token = [&](int r) { return tok0 + a.group.div((uint32_t)r); };
    int lim[RT];
    int lim_lo = 0x7fffffff, lim_hi = 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = r0 + 16 * t + j;
        lim[t] = 0;
        if (r < nrows) {
            const int tok = row_token(r), s = a.queries.div((uint32_t)tok);
            const int len = a.lens[s];
            const int n = len - a.n_qt + 1 + (tok - s * a.n_qt);
            lim[t] = len < 0 || len > a.max_len ? 0 : max(0, pre ? min(n, a.prefix_len) : n);
            if (lim[t] > (pre ? 0 : a.own_from)) lim_lo = min(lim_lo, lim[t]);   // (of rows that see some key here)
            lim_hi = max(lim_hi, lim[t]);
        }
    }
    lim_lo = __builtin_amdgcn_readfirstlane(row_min(lim_lo));
    lim_hi = __builtin_amdgcn_readfirstlane(-row_min(-lim_hi));

    // key tiles of this split: tiles [ta, tb) of the part's keys [k_lo, lim_hi)
    const int k_lo = pre ? 0 : a.own_from;
    const int t_first = k_lo / kAttnTile;
    const int t_end = lim_hi > k_lo ? (lim_hi + kAttnTile - 1) / kAttnTile : t_first;
    const int ntile = t_end - t_first;
    const int per = splits == 1 ? ntile : (pre ? a.div_p : a.splits_o).div((uint32_t)(ntile + splits - 1));
    const int ta = t_first + min(ntile, per * split), tb = t_first + min(ntile, per * (split + 1));

    // queries as the scores' B operand
    u32x4_t qv[RT][KS];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = r0 + 16 * t + j;
        const bool in = r < nrows;
        const int tok = in ? row_token(r) : 0;
        const int head = kvh * grp + (in ? r - (tok - tok0) * grp : 0);
        const uint8_t *qp = static_cast<const uint8_t *>(a.q) + 2 * ((int64_t)tok * a.ldq + (int64_t)head * D + 8 * g);
#pragma unroll
        for (int k = 0; k < KS; ++k)
            qv[t][k] = in ? *reinterpret_cast<const u32x4_t *>(qp + 64 * k) : u32x4_t{0u, 0u, 0u, 0u};
    }

    float4_t o[RT][DPL];
    float m[RT], ms[RT], l[RT];   // reference (-inf: none yet), the same as a number, sum of this lane
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = -__builtin_inff();
        ms[t] = 0.f;
        l[t] = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[t][e] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t *trow = a.table + (int64_t)seq * a.ld_table;
    const uint8_t *kbase = static_cast<const uint8_t *>(a.kc) + 2 * (int64_t)kvh * a.head_stride;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.vc) + 2 * (int64_t)kvh * a.head_stride;
    const int ts = (int)a.token_stride;
    const int psz = (int)a.page.d;

    u32x4_t kv[2][KS];
    uint32_t vv[8][VD];

    // element offset of key's row, and whether its page exists
    const auto key_row = [&](int key, bool &ok) {
        const int pi = a.page.div((uint32_t)key);
        const int page = (key < a.joint_len ? a.table : trow)[pi];
        ok = page >= 0 && page < a.n_pages;
        return (int64_t)(ok ? page : 0) * a.page_stride + (int64_t)(key - pi * psz) * a.token_stride;
    };
    // Where a tile's rows are: byte offsets of its halves (P16), or of every key in the wave's
    // lds_row.  Returns the keys whose page does not exist.
    int64_t base[2];
    const auto find_tile = [&](int tile) {
        const int key0 = tile * kAttnTile;
        uint32_t bad = 0;
        if constexpr (P16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // a half past the last seen key reads the first half again (it is masked)
                const int kk = key0 + 16 * h < lim_hi ? key0 + 16 * h : key0;
                bool ok;
                base[h] = 2 * key_row(kk, ok);
                if (!ok) bad |= 0xffffu << (16 * h);
            }
        } else {
            const int key = min(max(key0 + (lane & 31), k_lo), lim_hi - 1);
            bool ok;
            const int64_t row = 2 * key_row(key, ok);
            bad = (uint32_t)__ballot(!ok);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (lane < kAttnTile) lds_row[wave][lane] = row;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        return bad;
    };
    const auto load_k = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *kp = P16 ? kbase + base[h] + 2 * (j * ts + 8 * g) : kbase + lds_row[P16 ? 0 : wave][P16 ? 0 : 16 * h + j] + 16 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) kv[h][k] = *reinterpret_cast<const u32x4_t *>(kp + 64 * k);
        }
    };
    const auto load_v = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t *vp = P16 ? vbase + base[i / 4] + 2 * ((4 * g + i % 4) * ts + DPL * j)
                                    : vbase + lds_row[P16 ? 0 : wave][P16 ? 0 : 16 * (i / 4) + 4 * g + i % 4] + 2 * DPL * j;
            load_dwords<VD>(vp, vv[i]);
        }
    };
    // the value tile's operand of dim e: its 8 keys' halves
    const auto v_operand = [&](int e) {
        const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
        u32x4_t r;
#pragma unroll
        for (int p = 0; p < 4; ++p) r[p] = __builtin_amdgcn_perm(vv[2 * p + 1][e / 2], vv[2 * p][e / 2], sel);
        return r;
    };

    // This lane's part of a row tile's O in the wave's part of lds_o.
    const auto o_to_lds = [&](int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < DPL; e += 4)
                *reinterpret_cast<float4_t *>(&lds_o[wave][16 * t + j][DPL * (4 * g + i) + e]) =
                    float4_t{o[t][e][i], o[t][e + 1][i], o[t][e + 2][i], o[t][e + 3][i]};
    };
    const auto o_from_lds = [&](int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < DPL; e += 4) {
                const float4_t v = *reinterpret_cast<const float4_t *>(&lds_o[wave][16 * t + j][DPL * (4 * g + i) + e]);
#pragma unroll
                for (int q = 0; q < 4; ++q) o[t][e + q][i] = v[q];
            }
    };

    const auto scores = [&](float4_t (&sc)[RT][2]) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sc[t][h] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k) sc[t][h] = Mma<CT>::mul(kv[h][k], qv[t][k], sc[t][h]);
            }
    };
    // Scores to weights: masks, the running reference and sum, and P rounded.
    const auto softmax = [&](float4_t (&sc)[RT][2], u32x4_t (&p)[RT], int key0, bool edge, uint32_t bad) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float4_t(&s)[2] = sc[t];
            if (edge) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int kk = 16 * h + 4 * g + i;
                        if ((bad >> kk) & 1u) s[h][i] = __builtin_nanf("");
                        if (key0 + kk >= lim[t] || key0 + kk < k_lo) s[h][i] = -__builtin_inff();
                    }
            }
            const float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                                    fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3]))) *
                              a.scale2;
            if (__ballot(top > m[t] + 8.f)) {
                // raise the rows' references to their maxima so far and rescale what they hold
                float mx = fmaxf(m[t], top);
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float mn = mx == -__builtin_inff() ? 0.f : mx;
                const float f = m[t] == mx ? 1.f : __builtin_amdgcn_exp2f(m[t] - mn);
                m[t] = mx;
                ms[t] = mn;
                l[t] *= f;
#pragma unroll
                for (int e = 0; e < DPL; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][e][i] *= f;
            }
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 4][i % 4], a.scale2, -ms[t]));
                l[t] += w[i];
            }
            p[t] = u32x4_t{pack2<CT>(w[0], w[1]), pack2<CT>(w[2], w[3]), pack2<CT>(w[4], w[5]), pack2<CT>(w[6], w[7])};
        }
    };

    // Tiles from t_split on hold keys that only some of the rows see.
    const int t_split = lim_lo < lim_hi ? max(ta, min(tb, lim_lo / kAttnTile)) : tb;
    int tile = ta + wave;
    // The keys of the next tile are on their way while this one's softmax and values are worked
    // on, its values during the next scores: one set of registers each.
    uint32_t bad = 0, next_bad = 0;
    if (tile < t_split) {
        next_bad = find_tile(tile);
        load_k();
        load_v();
    }
    for (; tile < t_split; tile += W) {
        bad = next_bad;
        const bool more = tile + W < t_split;
        if (more) next_bad = find_tile(tile + W);
        const int key0 = tile * kAttnTile;
        const bool edge = key0 < k_lo || key0 + kAttnTile > lim_hi || bad != 0;   // some key needs a mask
        float4_t sc[RT][2];
        u32x4_t p[RT];
        scores(sc);
        if (more) load_k();
        softmax(sc, p, key0, edge, bad);
        if (edge) {     // what nobody sees may be NaN: its value rows go
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int kk = key0 + 16 * (i / 4) + 4 * g + i % 4;
                const bool seen = kk < lim_hi && kk >= k_lo;
#pragma unroll
                for (int q = 0; q < VD; ++q) vv[i][q] = seen ? vv[i][q] : 0u;
            }
        }
#pragma unroll
        for (int e = 0; e < DPL; ++e) {
            const u32x4_t va = v_operand(e);
#pragma unroll
            for (int t = 0; t < RT; ++t) o[t][e] = Mma<CT>::mul(va, p[t], o[t][e]);
        }
        if (more) load_v();
    }
    // The others, without overlap: a tile's values are multiplied once per distinct limit, lowest
    // first, with value rows at or past it zeroed; the rows of other limits take back what they had
    // (a zeroed P would not do: 0 * NaN reaches them).  The wave's part of lds_o holds it meanwhile.
    for (; tile < tb; tile += W) {
        bad = find_tile(tile);
        const int key0 = tile * kAttnTile;
        float4_t sc[RT][2];
        u32x4_t p[RT];
        load_k();
        scores(sc);
        softmax(sc, p, key0, true, bad);
        load_v();
        int done = max(key0, k_lo);             // (rows of limits up to here see nothing in this tile)
        while (true) {
            int cur = 0x7fffffff;
#pragma unroll
            for (int t = 0; t < RT; ++t)
                if (lim[t] > done) cur = min(cur, lim[t]);
            cur = __builtin_amdgcn_readfirstlane(row_min(cur));
            if (cur == 0x7fffffff) break;
            done = cur;
            uint32_t keep[4];                   // per pair of keys: which halves stay
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int k0 = key0 + 16 * (q / 2) + 4 * g + 2 * (q % 2);
                keep[q] = (k0 < cur && k0 >= k_lo ? 0xffffu : 0u) | (k0 + 1 < cur && k0 + 1 >= k_lo ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) o_to_lds(t);
#pragma unroll
            for (int e = 0; e < DPL; ++e) {
                u32x4_t va = v_operand(e);
#pragma unroll
                for (int q = 0; q < 4; ++q) va[q] &= keep[q];
#pragma unroll
                for (int t = 0; t < RT; ++t) o[t][e] = Mma<CT>::mul(va, p[t], o[t][e]);
            }
            settle();
#pragma unroll
            for (int t = 0; t < RT; ++t)
                if (lim[t] != cur) o_from_lds(t);
        }
    }

    // join the waves' results
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if (lim[t] <= k_lo || m[t] == -__builtin_inff()) {   // no key seen: what was added up is not data
            m[t] = -__builtin_inff();
            l[t] = 0.f;
#pragma unroll
            for (int e = 0; e < DPL; ++e) o[t][e] = float4_t{0.f, 0.f, 0.f, 0.f};
        }
        float lt = l[t];
        lt += __shfl_xor(lt, 16);
        lt += __shfl_xor(lt, 32);
        if (g == 0) {
            lds_m[wave][16 * t + j] = m[t];
            lds_l[wave][16 * t + j] = lt;
        }
        o_to_lds(t);
    }
    __syncthreads();
    const int rows_here = min(nrows - r0, RT * 16);
    const int nsplit = a.splits_p + (a.wgs_o ? (int)a.splits_o.d : 0);
    const int sidx = pre ? split : a.splits_p + split;
#pragma unroll 1
    for (int x = tid; x < rows_here * (D / 4); x += 64 * W) {
        const int r = x / (D / 4), d = 4 * (x % (D / 4));
        float mm = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < W; ++w) mm = fmaxf(mm, lds_m[w][r]);
        const float mb = mm == -__builtin_inff() ? 0.f : mm;
        float ll = 0.f;
        float4_t oo = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int w = 0; w < W; ++w) {
            const float f = __builtin_amdgcn_exp2f(lds_m[w][r] - mb);
            ll = __builtin_fmaf(f, lds_l[w][r], ll);
            const float4_t v = *reinterpret_cast<const float4_t *>(&lds_o[w][r][d]);
#pragma unroll
            for (int i = 0; i < 4; ++i) oo[i] = __builtin_fmaf(f, v[i], oo[i]);
        }
        const int tok = row_token(r0 + r);
        const int head = kvh * grp + (r0 + r - (tok - tok0) * grp);
        if (nsplit == 1) {
            const int len = a.lens[a.queries.div((uint32_t)tok)];
            const float nv = len < 0 || len > a.max_len ? __builtin_nanf("") : 0.f;
            const float inv = 1.f / ll;
            float4_t res;
#pragma unroll
            for (int i = 0; i < 4; ++i) res[i] = ll == 0.f ? nv : oo[i] * inv;
            CT *op = static_cast<CT *>(a.out) + (int64_t)tok * a.ldo + (int64_t)head * D + d;
            *reinterpret_cast<u32x2_t *>(op) = u32x2_t{pack2<CT>(res[0], res[1]), pack2<CT>(res[2], res[3])};
        } else {
            const int64_t row = ((int64_t)tok * a.n_q + head) * nsplit + sidx;
            *reinterpret_cast<float4_t *>(a.part_o + row * D + d) = oo;
            if (d == 0) *reinterpret_cast<float2_t *>(a.part_ml + 2 * row) = float2_t{mm, ll};
        }
    }
}

// Joins the splits (at most 64) of a row: a workgroup per row, D/4 lanes for a split's O.
template <typename CT, int D>
__global__ __launch_bounds__(256) void attn_join(AttnShared a, int nsplit) {
    constexpr int L = D / 4, G = 256 / L;
    __shared__ float4_t lds[256];
    __shared__ float lds_f[64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x;
    // every wave: the splits' weights, one a lane
    float2_t ml = {-__builtin_inff(), 0.f};
    if (lane < nsplit) ml = *reinterpret_cast<const float2_t *>(a.part_ml + 2 * (row * nsplit + lane));
    float mm = ml.x;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) mm = fmaxf(mm, __shfl_xor(mm, off));
    const float f = __builtin_amdgcn_exp2f(ml.x - (mm == -__builtin_inff() ? 0.f : mm));
    float ll = f * ml.y;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) ll += __shfl_xor(ll, off);
    if (tid < 64) lds_f[lane] = f;
    __syncthreads();
    const int d = 4 * (tid % L);
    float4_t oo = {0.f, 0.f, 0.f, 0.f};
    const float *po = a.part_o + row * nsplit * D + d;
#pragma unroll 4
    for (int s = tid / L; s < nsplit; s += G) {
        const float w = lds_f[s];
        const float4_t v = *reinterpret_cast<const float4_t *>(po + s * D);
#pragma unroll
        for (int i = 0; i < 4; ++i) oo[i] = __builtin_fmaf(w, v[i], oo[i]);
    }
    lds[tid] = oo;
    __syncthreads();
    if (tid < L) {
#pragma unroll
        for (int k = 1; k < G; ++k) {
            const float4_t v = lds[k * L + tid];
#pragma unroll
            for (int i = 0; i < 4; ++i) oo[i] += v[i];
        }
        const int tok = (int)(row / a.n_q), head = (int)(row - (int64_t)tok * a.n_q);
        const int len = a.lens[a.queries.div((uint32_t)tok)];
        const float nv = len < 0 || len > a.max_len ? __builtin_nanf("") : 0.f;
        const float inv = 1.f / ll;
        float4_t res;
#pragma unroll
        for (int i = 0; i < 4; ++i) res[i] = ll == 0.f ? nv : oo[i] * inv;
        CT *op = static_cast<CT *>(a.out) + (int64_t)tok * a.ldo + (int64_t)head * D + d;
        *reinterpret_cast<u32x2_t *>(op) = u32x2_t{pack2<CT>(res[0], res[1]), pack2<CT>(res[2], res[3])};
    }
}

// 8 waves where two of them fit a SIMD's registers with one row tile each
constexpr int attn_waves(int64_t dim, int row_tiles) { return row_tiles == 1 && dim < 256 ? 8 : 4; }

AttnPlan attn_plan(int64_t n_seqs, int64_t n_q, int64_t n_kv, int64_t dim, int64_t n_qt, int64_t prefix_len,
                   int64_t max_len) {
    AttnPlan p{};
    const int64_t rows_o = n_qt * (n_q / n_kv), rows_p = n_seqs * rows_o;
    const auto tiles = [](int64_t keys) { return (keys + kAttnTile - 1) / kAttnTile; };
    const auto groups = [&](int64_t rows) { return (rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles); };
    // enough workgroups for the chip, but two tiles for each of a workgroup's waves
    const auto splits = [&](int64_t units, int64_t t) {
        int64_t s = (512 + units - 1) / units;
        if (s > t / (2 * p.waves)) s = t / (2 * p.waves);
        if (s > kAttnMaxSplits) s = kAttnMaxSplits;
        return s < 1 ? (int64_t)1 : s;
    };
    // Short and few: one workgroup per sequence and key head takes all keys, prefix included
    // (read once per sequence, from the L2), and writes the result itself: no join.
    const int big = dim == 256 ? 1 : 2;
    p.row_tiles = rows_o <= 16 ? 1 : big;
    p.waves = attn_waves(dim, p.row_tiles);
    p.joint = prefix_len > 0 && tiles(max_len) <= 5 * p.waves && n_seqs * n_kv * groups(rows_o) <= 256;
    const bool shared = prefix_len > 0 && !p.joint;
    if (shared) {
        p.row_tiles = rows_p <= 16 ? 1 : big;
        p.waves = attn_waves(dim, p.row_tiles);
    }
    p.groups_p = groups(rows_p);
    p.groups_o = groups(rows_o);
    p.splits_p = shared ? splits(p.groups_p * n_kv, tiles(prefix_len)) : 0;
    const int64_t own = shared ? tiles(max_len) - prefix_len / kAttnTile : tiles(max_len);
    p.splits_o = !shared || max_len > prefix_len ? (own <= 5 * p.waves ? 1 : splits(n_seqs * p.groups_o * n_kv, own)) : 0;
    const int64_t n = p.splits_p + p.splits_o;
    p.ws_bytes = n <= 1 ? 0 : (size_t)(n * rows_p * n_kv) * (size_t)(dim + 2) * 4;
    return p;
}

hipError_t launch_attn_shared(AttnShared a, const AttnPlan &p, Act ct, int dim, hipStream_t s) {
    const auto div = [](int64_t d) { return FastDiv::make((uint32_t)(d > 0 ? d : 1)); };
    a.groups_p = div(p.groups_p);
    a.groups_o = div(p.groups_o);
    a.heads = div(a.n_kv);
    a.queries = div(a.n_qt);
    a.div_p = div(p.splits_p);
    a.splits_o = div(p.splits_o);
    a.splits_p = (int)p.splits_p;
    a.rows_o = a.n_qt * (int)a.group.d;
    a.rows_p = a.n_seqs * a.rows_o;
    a.own_from = p.joint ? 0 : a.prefix_len;
    a.joint_len = p.joint ? a.prefix_len : 0;
    const int64_t units_p = a.n_kv * p.splits_p;
    a.xcd_p = p.groups_p > 1 && units_p % 8 == 0;
    a.wgs_p = (int)(p.groups_p * units_p);
    a.wgs_o = (int)(p.groups_o * a.n_kv * p.splits_o * a.n_seqs);
    const int64_t n_out = (int64_t)a.rows_p * a.n_kv;
    const int nsplit = (int)(p.splits_p + p.splits_o);
    a.part_ml = a.part_o + nsplit * n_out * dim;
    const dim3 grid((unsigned)(a.wgs_p + a.wgs_o));
    const bool p16 = a.page.d % 16 == 0 && (!p.joint || a.prefix_len % 16 == 0);
    auto run = [&](auto ctag, auto d, auto rt) -> hipError_t {
        using CT = decltype(ctag);
        constexpr int D = decltype(d)::value, RT = decltype(rt)::value, W = attn_waves(D, RT);
        if (p16) attn_rows<CT, D, RT, W, true><<<grid, 64 * W, 0, s>>>(a);
        else attn_rows<CT, D, RT, W, false><<<grid, 64 * W, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || nsplit == 1) return e;
        attn_join<CT, D><<<dim3((unsigned)n_out), 256, 0, s>>>(a, nsplit);
        return hipGetLastError();
    };
    auto by_rt = [&](auto ctag, auto d) -> hipError_t {
        constexpr int big = decltype(d)::value == 256 ? 1 : 2;
        if (p.row_tiles == 1) return run(ctag, d, std::integral_constant<int, 1>{});
        return run(ctag, d, std::integral_constant<int, big>{});
    };
    auto by_dim = [&](auto ctag) -> hipError_t {
        if (dim == 64) return by_rt(ctag, std::integral_constant<int, 64>{});
        if (dim == 128) return by_rt(ctag, std::integral_constant<int, 128>{});
        return by_rt(ctag, std::integral_constant<int, 256>{});
    };
    return ct == Act::F16 ? by_dim(_Float16{}) : by_dim(bf16_t{});
}

}  // namespace q2_0
