// Attention of a batch over a paged cache, the prefix that the sequences share read once.
//
//   o[r] = sum_i p_ri v_i / sum_i p_ri,   p_ri = 2^(c q_r.k_i - m_r),   c = scale log2 e
//
// The softmax is one pass: a wave keeps a reference exponent m_r, the sum l_r and the
// unnormalised O_r (f32) of its rows; two results over different keys join as
// l = l1 2^(m1-m) + l2 2^(m2-m), O likewise, with m = max(m1, m2).
//
// Operands.  32 keys at a time:
//  * S^T = K Q^T (v_mfma 16x16x32): A = 16 keys x 32 dims, 16 bytes a lane, as they lie in
//    the cache; B = Q^T, loaded once.  D: lane (row j = lane%16, g = lane/16) holds the
//    scores of keys 4g..4g+3 of each 16-key half for row j.
//  * O^T += V^T P^T: B = P^T needs, in lane (j, g), 8 keys of row j: exactly the two
//    halves' scores of that lane, as two operands: the weight rounded to 16 bits and what that left, again
//    in 16 bits.  With the first alone results erred 1.4 times as much as with weights in f32 (relative to
//    64 bits 2.3e-3 against 1.65e-3 in bfloat16, whose own rounding is most of that), and the difference of
//    nearly equal weights was lost; with both the two err alike, for half as many matrix
//    instructions again (64 sequences over 32768 keys 77 -> 87 us, 16 over 4096 15.9 -> 16.5, one of 777 11.1 -> 11.5).
//    A = V^T takes the same 8 keys {4g+i, 16+4g+i} of
//    16 dims per MFMA e (c = lane%16): d = DPL*c + e in the own part, where a lane holds DPL
//    consecutive dims of those 8 value rows and pairs keys up with one v_perm_b32 a dword, and
//    d = 16 e + c in the prefix part, which reads them transposed from LDS.
//  * l += 1 P^T, two more MFMAs: the sum takes the same operands as the values.
// So a score never leaves its lane: no lane exchange per step.  The reference m_r is only
// raised when some score passes it by a headroom (a ballot decides), for which f32 and P have room.
// f16 has no room below: weights under 2^-25 would be lost, which tens of thousands of keys behind a
// leading one add up to (30000 of them at 2^-26 are 4e-4 of the sum).  So its weights carry a factor 2^11, in O and l
// alike, which puts their last place at 2^-35 of the reference's, and the headroom is 2^4.
//
// A key head's rows are (query token, query head of its group).  Two parts, one launch:
//  * own keys (own_part): a workgroup takes up to 16 rows of one sequence; its waves take
//    different key tiles, straight from the cache into operand registers (full 256-byte value
//    rows, 64-byte pieces of key rows), the next tile's keys on their way during the softmax and
//    its values during the next scores.  HBM-bound with enough sequences.
//  * the prefix (prefix_part), where the rows of all sequences stand together: the waves take
//    different rows (16 RTP each) of the same key tiles, which go to LDS once per workgroup by
//    16-byte LDS-DMA loads, two tiles ahead, one barrier a tile.  A key row's 16-byte pieces
//    sit XOR-swizzled by its number, so that the 16 rows of an operand read meet 16 different
//    bank groups; values sit so that a transposing read's 4 rows x 16 dims are 128 bytes in a row.
//    (Key operands straight from the cache touch 64 lines an instruction, 16 rows
//    x 4 pieces: with every wave reading them so, the L1's tag rate held 64 sequences over
//    32768 keys at 123 us.)  Of 32 keys x 32 rows ~120
//    VALU and 52 matrix instructions: bound by issue with two workgroups on a CU (1.6 us a tile for both, 128
//    dims and 128 rows), by the latency of a tile's steps with one (1.1).
//    Few rows, or a short prefix of few sequences, go the own part's way instead.
// Workgroups that read the same prefix keys for other rows get launch numbers 8 apart: the same XCD, whose
// L2 then serves all but one of them (64 sequences over 8192 keys, four row groups: 55 us spread over the XCDs, 50 so).
// Splits of the key axis join in attn_join.
//
// Masks.  A row sees keys below its limit.  Scores past it become -inf before the maximum, value
// rows nobody sees are zeroed, and tiles whose keys only some of a wave's rows see (draft tokens,
// sequences shorter than the prefix) go through a loop of their own, so that what lies in
// unseen places (NaN, inf) reaches no row that does not see it.  Addresses are clamped to seen keys.
#include <type_traits>

#include "layer_common.h"
#include "lds_dma.h"

namespace q2_0 {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));

template <typename CT>
struct Mma;
template <>
struct Mma<_Float16> {
    static constexpr uint32_t kOnes = 0x3c003c00u;
    static constexpr float kHead = 4.f, kBias = 11.f;     // of the weights, as powers of two; together at most 15
    static constexpr float kOver = 1.f + 0x1p-11f;
    static __device__ __forceinline__ float4_t mul(u32x4_t a, u32x4_t b, float4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c,
                                                      0, 0, 0);
    }
};
template <>
struct Mma<bf16_t> {
    static constexpr uint32_t kOnes = 0x3f803f80u;
    static constexpr float kHead = 8.f, kBias = 0.f;
    static constexpr float kOver = 1.f + 0x1p-8f;
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
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false);
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

// Waves of a workgroup: 4, so that two workgroups share a CU and are not in step (one's softmax then runs
// beside the other's matrix instructions), and a sequence's keys split finely.  In us with 4 and with 8 (8 key heads
// of 128): 1200 keys of one sequence 9.7 and 12.0, 2000 9.9 and 13.0, 16 sequences of 2000 30.0 and 36.0; where keys
// are not split 8 gain a little, 777 keys of one sequence 11.5 and 10.9, of 16 14.0 and 13.0.
constexpr int kAttnWaves = 4;

// The page table through the scalar cache (uniform index).
__device__ __forceinline__ int table_at(const int32_t *t, int i) {
    typedef const __attribute__((address_space(4))) int32_t *ConstPtr;
    return ((ConstPtr)(uintptr_t)t)[i];
}

// Softmax weights of 8 keys for a row, as the second product takes them: the weight in the cache's type and what
// that rounding left, again in that type.  All weights are carried kOver times as large, in the second operand, so that
// this one is above 0 where the first is: with both signs, or 0, an infinite value would come out as NaN.
struct Weights {
    u32x4_t hi, lo;
};

template <typename CT>
__device__ __forceinline__ float2_t unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2_t unpack2<_Float16>(uint32_t v) {
    const half2_t h = __builtin_bit_cast(half2_t, v);
    return float2_t{(float)h.x, (float)h.y};
}
template <>
__device__ __forceinline__ float2_t unpack2<bf16_t>(uint32_t v) {
    return float2_t{__builtin_bit_cast(float, v << 16), __builtin_bit_cast(float, v & 0xffff0000u)};
}

// What a wave knows of its rows, RT tiles of 16, and holds of their results.
template <typename CT, int D, int RT>
struct Rows {
    static constexpr int KS = D / 32;       // 32-dim steps of a score
    static constexpr int DPL = D / 16;      // dims per lane of a value row
    static constexpr int VD = DPL / 2;      // dwords of those
    static constexpr int OS = D + 4;        // LDS floats per row

    u32x4_t q[RT][KS];       // queries as the scores' B operand
    float4_t o[RT][DPL];
    float m[RT], ms[RT];     // reference (-inf: none yet); the weights' exponents are relative to ms
    float4_t l[RT];          // row j's sum, four times
    int lim[RT];             // keys row j sees
    int lim_lo, lim_hi;      // the least (of rows that see some key past k_lo) and most of the wave's rows
    u32x4_t k[2][KS];        // a key tile's operands
    uint32_t v[8][VD];       // and its value rows

    // Rows r0 .. of nrows; tok0: the first row's query row; key head kvh.
    __device__ __forceinline__ void init(const AttnShared &a, int r0, int nrows, int tok0, int kvh, int k_lo, int k_hi, int j, int g) {
        const int grp = (int)a.group.d;
        lim_lo = 0x7fffffff, lim_hi = 0;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = r0 + 16 * t + j;
            lim[t] = 0, m[t] = -__builtin_inff(), ms[t] = 0.f, l[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < DPL; ++e) o[t][e] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; ++s) q[t][s] = u32x4_t{0u, 0u, 0u, 0u};
            if (r < nrows) {
                const int tr = a.group.div((uint32_t)r), tok = tok0 + tr, s = a.queries.div((uint32_t)tok);
                const int len = a.lens[s];
                const int n = min(k_hi, len - a.n_qt + 1 + (tok - s * a.n_qt));
                lim[t] = len < 0 || len > a.max_len ? 0 : max(0, n);
                if (lim[t] > k_lo) lim_lo = min(lim_lo, lim[t]);
                lim_hi = max(lim_hi, lim[t]);
                const uint8_t *qp = static_cast<const uint8_t *>(a.q) +
                                    2 * ((int64_t)tok * a.ldq + (int64_t)(kvh * grp + r - tr * grp) * D + 8 * g);
#pragma unroll
                for (int st = 0; st < KS; ++st) q[t][st] = *reinterpret_cast<const u32x4_t *>(qp + 64 * st);
            }
        }
        lim_lo = __builtin_amdgcn_readfirstlane(row_min(lim_lo));
        lim_hi = __builtin_amdgcn_readfirstlane(-row_min(-lim_hi));
    }
    __device__ __forceinline__ void scores(float4_t (&s)[2], int t) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < KS; ++i) s[h] = Mma<CT>::mul(k[h][i], q[t][i], s[h]);
        }
    }
    // What row j does not see, and NaN for keys whose page does not exist (bad)
    __device__ __forceinline__ void mask(float4_t (&s)[2], int t, int key0, int k_lo, uint32_t bad, int g) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int kk = 16 * h + 4 * g + i;
                if ((bad >> kk) & 1u) s[h][i] = __builtin_nanf("");
                if (key0 + kk >= lim[t] || key0 + kk < k_lo) s[h][i] = -__builtin_inff();
            }
    }
    // Where a score passes its row's reference by 2^kHead: raises the rows' references to their maxima so far
    // and rescales what they hold.
    __device__ __forceinline__ void raise(const float4_t (&s)[2], int t, float scale2) {
        const float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                                fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3]))) *
                          scale2;
        if (__ballot(top > m[t] + Mma<CT>::kHead)) {
            float mx = fmaxf(m[t], top);
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = mx == -__builtin_inff() ? 0.f : mx - Mma<CT>::kBias;
            const float f = m[t] == mx ? 1.f : __builtin_amdgcn_exp2f(m[t] == -__builtin_inff() ? m[t] : ms[t] - mn);
            m[t] = mx;
            ms[t] = mn;
#pragma unroll
            for (int i = 0; i < 4; ++i) l[t][i] *= f;
#pragma unroll
            for (int e = 0; e < DPL; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][e][i] *= f;
        }
    }
    // Scores to weights P, as two operands of the matrix cores.
    __device__ __forceinline__ Weights weights(const float4_t (&s)[2], int t, float scale2) {
        Weights p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) w[h] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 2][2 * (i % 2) + h], scale2, -ms[t]));
            const uint32_t hi = pack2<CT>(w[0], w[1]);
            const float2_t r = unpack2<CT>(hi);
            p.hi[i] = hi;
            p.lo[i] = pack2<CT>(__builtin_fmaf(w[0], Mma<CT>::kOver, -r.x), __builtin_fmaf(w[1], Mma<CT>::kOver, -r.y));
        }
        return p;
    }
    // the value tile's operand of dim e: its 8 keys' halves
    __device__ __forceinline__ u32x4_t v_operand(int e) const {
        const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
        u32x4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_perm(v[2 * i + 1][e / 2], v[2 * i][e / 2], sel);
        return r;
    }
    // Which halves of a value operand's four dwords are keys in [k_lo, end)
    static __device__ __forceinline__ u32x4_t keys_kept(int key0, int k_lo, int end, int g) {
        u32x4_t keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k0 = key0 + 16 * (i / 2) + 4 * g + 2 * (i % 2);
            keep[i] = (k0 < end && k0 >= k_lo ? 0xffffu : 0u) | (k0 + 1 < end && k0 + 1 >= k_lo ? 0xffff0000u : 0u);
        }
        return keep;
    }
    // l += P 1, from the same operands as the values' sum.
    __device__ __forceinline__ void sums(const Weights &p, int t) {
        constexpr uint32_t one = Mma<CT>::kOnes;
        const u32x4_t ones = {one, one, one, one};
        l[t] = Mma<CT>::mul(ones, p.lo, Mma<CT>::mul(ones, p.hi, l[t]));
    }
    // O += P V; va[e]: the operands
    __device__ __forceinline__ void values(const Weights (&p)[RT], const u32x4_t (&va)[DPL]) {
#pragma unroll
        for (int t = 0; t < RT; ++t) sums(p[t], t);
#pragma unroll
        for (int e = 0; e < DPL; ++e)
#pragma unroll
            for (int t = 0; t < RT; ++t) o[t][e] = Mma<CT>::mul(va[e], p[t].hi, o[t][e]);
#pragma unroll
        for (int e = 0; e < DPL; ++e)
#pragma unroll
            for (int t = 0; t < RT; ++t) o[t][e] = Mma<CT>::mul(va[e], p[t].lo, o[t][e]);
    }
    // Row tile t's O in a wave's LDS area of 16 rows; an operand's dims are DPL apart, or 16 in a row (ROW16).
    template <bool ROW16>
    __device__ __forceinline__ void o_to_lds(float *area, int t, int j, int g) const {
        if constexpr (ROW16) {
#pragma unroll
            for (int e = 0; e < DPL; ++e) *reinterpret_cast<float4_t *>(area + j * OS + 16 * e + 4 * g) = o[t][e];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < DPL; e += 4)
                    *reinterpret_cast<float4_t *>(area + j * OS + DPL * (4 * g + i) + e) =
                        float4_t{o[t][e][i], o[t][e + 1][i], o[t][e + 2][i], o[t][e + 3][i]};
        }
    }
    // A tile whose keys only some rows see (its keys in k): its values are multiplied once per distinct limit
    // inside it, and once for all rows that see it whole, lowest first, with value rows at or past the limit zeroed,
    // and only the rows of that limit take the product
    // (a zeroed P would not do: 0 * NaN reaches the others).  Nothing in the loop branches by lane: a
    // branch on lim == cur was carried into the next pass by the compiler, whose minimum over the rows
    // then missed lanes and never came to an end.
    template <typename Operand>
    __device__ __forceinline__ void mixed_tile(int t, float scale2, int key0, int k_lo, uint32_t bad, int g, const Operand &operand) {
        float4_t s[2];
        scores(s, t);
        settle();
        mask(s, t, key0, k_lo, bad, g);
        raise(s, t, scale2);
        const Weights p = weights(s, t, scale2);
        sums(p, t);
        int done = max(key0, k_lo);             // (rows of limits up to here see nothing in this tile)
        const int mylim = min(lim[t], key0 + kAttnTile);
#pragma unroll 1
        for (int pass = 0; pass < 16; ++pass) { // (16 rows: no more limits)
            const int cur = __builtin_amdgcn_readfirstlane(row_min(mylim > done ? mylim : 0x7fffffff));
            if (cur == 0x7fffffff) break;
            done = cur;
            const u32x4_t keep = keys_kept(key0, k_lo, cur, g);
            const bool mine = mylim == cur;
#pragma unroll
            for (int e = 0; e < DPL; ++e) {
                u32x4_t va = operand(e);
#pragma unroll
                for (int i = 0; i < 4; ++i) va[i] &= keep[i];
                const float4_t r = Mma<CT>::mul(va, p.lo, Mma<CT>::mul(va, p.hi, float4_t{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][e][i] = mine ? o[t][e][i] + r[i] : o[t][e][i];
            }
        }
        settle();
    }
    // Row j's final reference, which its weights were relative to, and sum; rows that saw nothing hold nothing (a
    // row that saw nothing but NaN has no reference either, and keeps its NaN).
    __device__ __forceinline__ void finish(int k_lo) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (lim[t] <= k_lo) {
                m[t] = -__builtin_inff();
                l[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < DPL; ++e) o[t][e] = float4_t{0.f, 0.f, 0.f, 0.f};
            }
            if (m[t] != -__builtin_inff()) m[t] = ms[t];
        }
    }
};

// Two 16-byte LDS-DMA loads per lane (lds_dma.h, the wait after a write of M0 too) to kilobytes step apart, with a uniform
// base and a byte offset per lane.
__device__ __forceinline__ void lds_dma16x2(const void *base, uint32_t off0, uint32_t off1, uint32_t lds, uint32_t step) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %4\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %3\n\t"
        "s_add_u32 m0, m0, %5\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %2, %3\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(off0), "v"(off1), "s"(base), "s"(lds), "s"(step)
        : "memory", "scc");
}

// 4 rows x 16 elements from LDS, the lanes of a 16-lane group 8 bytes each along the rows (lane l: row l / 4);
// lane l gets element l of the four rows.
__device__ __forceinline__ u32x2_t read_transposed(const uint8_t *p) {
    typedef short Four __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) Four *LdsPtr;
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p)));
}

// Stands for rows of pages that do not exist: NaN in either type.
__device__ const uint32_t kNanRow[4] = {0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu};

// Where a key tile's rows are.  P16: the 16 keys of a half tile lie in one page (page_size % 16 == 0, and
// the keys of a half are all of one table row), whose number is read once for the wave: byte
// offsets of the halves.  Otherwise 32 lanes look up a key each and pass the rows round through
// the wave's lds_row.
template <typename CT, int D, bool P16>
struct KeyTile {
    const AttnShared &a;
    const int32_t *trow;        // the sequence's table row; keys below a.joint_len are in row 0
    const uint8_t *kbase, *vbase;
    int64_t *lds_row;
    int64_t base[2];

    __device__ __forceinline__ int64_t row_of(int key, int page, int pi, bool &ok) const {
        ok = page >= 0 && page < a.n_pages;
        return 2 * ((int64_t)(ok ? page : 0) * a.page_stride + (int64_t)(key - pi * (int)a.page.d) * a.token_stride);
    }
    __device__ __forceinline__ const int32_t *table_of(int key) const { return key < a.joint_len ? a.table : trow; }

    // keys key0 .. key0 + 31 (those outside [k_lo, k_hi) are not looked up); returns the keys whose page
    // does not exist
    __device__ __forceinline__ uint32_t find(int key0, int k_lo, int k_hi, int lane) {
        uint32_t bad = 0;
        if constexpr (P16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // a half past the last seen key reads the first half again (it is masked)
                const int kk = key0 + 16 * h < k_hi ? key0 + 16 * h : key0;
                const int pi = a.page.div((uint32_t)kk);
                bool ok;
                base[h] = row_of(kk, table_at(table_of(kk), pi), pi, ok);
                if (!ok) bad |= 0xffffu << (16 * h);
            }
        } else {
            const int key = min(max(key0 + (lane & 31), k_lo), k_hi - 1);
            const int pi = a.page.div((uint32_t)key);
            bool ok;
            const int64_t row = row_of(key, table_of(key)[pi], pi, ok);
            bad = (uint32_t)__ballot(!ok);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (lane < kAttnTile) lds_row[lane] = row;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        return bad;
    }
    // byte offset of row r of the tile
    __device__ __forceinline__ int64_t row(int r) const {
        if constexpr (P16) return (r < 16 ? base[0] : base[1]) + 2 * (r & 15) * (int)a.token_stride;
        else return lds_row[r];
    }
    template <int RT>
    __device__ __forceinline__ void load_k(Rows<CT, D, RT> &w, int j, int g) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t *p = P16 ? kbase + base[h] + 2 * (j * (int)a.token_stride + 8 * g) : kbase + lds_row[16 * h + j] + 16 * g;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) w.k[h][s] = *reinterpret_cast<const u32x4_t *>(p + 64 * s);
        }
    }
    template <int RT>
    __device__ __forceinline__ void load_v(Rows<CT, D, RT> &w, int j, int g) const {
        constexpr int DPL = D / 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t *p = P16 ? vbase + base[i / 4] + 2 * ((4 * g + i % 4) * (int)a.token_stride + DPL * j)
                                   : vbase + lds_row[16 * (i / 4) + 4 * g + i % 4] + 2 * DPL * j;
            load_dwords<DPL / 2>(p, w.v[i]);
        }
    }
};

// Result or partial of a row (output row tok, head): dims d .. d + 3 of split sidx.
template <typename CT, int D>
__device__ __forceinline__ void store_row(const AttnShared &a, int nsplit, int sidx, int tok, int head, int d, float4_t o, float m, float l) {
    if (nsplit == 1) {
        const int len = a.lens[a.queries.div((uint32_t)tok)];
        const float nv = len < 0 || len > a.max_len ? __builtin_nanf("") : 0.f;
        const float inv = 1.f / l;
        float4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = l == 0.f ? nv : o[i] * inv;
        CT *op = static_cast<CT *>(a.out) + (int64_t)tok * a.ldo + (int64_t)head * D + d;
        *reinterpret_cast<u32x2_t *>(op) = u32x2_t{pack2<CT>(r[0], r[1]), pack2<CT>(r[2], r[3])};
    } else {
        const int64_t row = ((int64_t)tok * a.n_q + head) * nsplit + sidx;
        *reinterpret_cast<float4_t *>(a.part_o + row * D + d) = o;
        if (d == 0) *reinterpret_cast<float2_t *>(a.part_ml + 2 * row) = float2_t{m, l};
    }
}

// LDS of attn_rows: the waves' O areas and joint references of the own part, or the prefix part's tile
// buffers (then its O areas); and the row tables.
template <int D, bool PRE>
struct AttnLds {
    static constexpr int W = kAttnWaves, OS = D + 4;
    static constexpr int kTileBytes = kAttnTile * D * 2;                   // keys of a tile
    static constexpr int kBlock = 1024 + (D == 64 ? 0 : D == 128 ? 128 : 64);       // a kilobyte of values, apart for the banks
    static constexpr int kValueBytes = kAttnTile * D * 2 / 1024 * kBlock;
    union {
        float o[W][16][OS];
        struct {
            __attribute__((aligned(16))) uint8_t k[3][PRE ? kTileBytes : 16], v[3][PRE ? kValueBytes : 16];
        } ring;
    };
    float m[W][16], l[W][16];
    int64_t row[W][kAttnTile];
    int least[W], most[W];
};

// One sequence's own keys (or all keys, prefix included, of a joint plan): waves take different tiles.
template <typename CT, int D, bool PRE, bool P16>
__device__ __forceinline__ void own_part(const AttnShared &a, AttnLds<D, PRE> &lds, int id, int tid) {
    constexpr int W = kAttnWaves;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), j = lane & 15, g = lane >> 4;
    int u = a.groups_o.div((uint32_t)id);
    const int rg = id - u * (int)a.groups_o.d;
    const int v = a.heads.div((uint32_t)u), kvh = u - v * a.n_kv;
    const int seq = a.splits_o.div((uint32_t)v), split = v - seq * (int)a.splits_o.d;
    const int splits = (int)a.splits_o.d, r0 = rg * 16, tok0 = seq * a.n_qt, k_lo = a.own_from;

    Rows<CT, D, 1> w;
    w.init(a, r0, a.rows_o, tok0, kvh, k_lo, 0x7fffffff, j, g);
    // key tiles of this split: tiles [ta, tb) of the keys [k_lo, lim_hi)
    const int t_first = k_lo / kAttnTile;
    const int ntile = max(0, (w.lim_hi > k_lo ? (w.lim_hi + kAttnTile - 1) / kAttnTile : t_first) - t_first);
    const int per = a.splits_o.div((uint32_t)(ntile + splits - 1));
    const int ta = t_first + min(ntile, per * split), tb = t_first + min(ntile, per * (split + 1));
    // tiles from t_split on hold keys that only some of the rows see
    const int t_split = w.lim_lo < w.lim_hi ? max(ta, min(tb, w.lim_lo / kAttnTile)) : tb;

    KeyTile<CT, D, P16> kt{a, a.table + (int64_t)seq * a.ld_table, static_cast<const uint8_t *>(a.kc) + 2 * (int64_t)kvh * a.head_stride,
                           static_cast<const uint8_t *>(a.vc) + 2 * (int64_t)kvh * a.head_stride, lds.row[wave], {0, 0}};
    int tile = ta + wave;
    uint32_t next_bad = 0;
    if (tile < t_split) {
        next_bad = kt.find(tile * kAttnTile, k_lo, w.lim_hi, lane);
        kt.load_k(w, j, g);
        kt.load_v(w, j, g);
    }
    for (; tile < t_split; tile += W) {
        const uint32_t bad = next_bad;
        const bool more = tile + W < t_split;
        if (more) next_bad = kt.find((tile + W) * kAttnTile, k_lo, w.lim_hi, lane);
        const int key0 = tile * kAttnTile;
        const bool edge = key0 < k_lo || key0 + kAttnTile > w.lim_hi || bad != 0;   // some key needs a mask
        float4_t s[2];
        Weights p[1];
        u32x4_t va[D / 16];
        w.scores(s, 0);
        if (more) kt.load_k(w, j, g);
        if (edge) w.mask(s, 0, key0, k_lo, bad, g);
        w.raise(s, 0, a.scale2);
        p[0] = w.weights(s, 0, a.scale2);
#pragma unroll
        for (int e = 0; e < D / 16; ++e) va[e] = w.v_operand(e);
        if (edge) {           // what nobody sees may be NaN
            const u32x4_t keep = w.keys_kept(key0, k_lo, w.lim_hi, g);
#pragma unroll
            for (int e = 0; e < D / 16; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) va[e][i] &= keep[i];
        }
        w.values(p, va);
        if (more) kt.load_v(w, j, g);
    }
    for (; tile < tb; tile += W) {
        const int key0 = tile * kAttnTile;
        const uint32_t bad = kt.find(key0, k_lo, w.lim_hi, lane);
        kt.load_k(w, j, g);
        kt.load_v(w, j, g);
        w.mixed_tile(0, a.scale2, key0, k_lo, bad, g, [&](int e) { return w.v_operand(e); });
    }
    // join the waves' results
    w.finish(k_lo);
    if (g == 0) {
        lds.m[wave][j] = w.m[0];
        lds.l[wave][j] = w.l[0][0];
    }
    w.template o_to_lds<false>(&lds.o[wave][0][0], 0, j, g);
    __syncthreads();
    const int grp = (int)a.group.d, rows_here = min(a.rows_o - r0, 16);
    const int nsplit = a.splits_p + splits;
#pragma unroll 1
    for (int x = tid; x < rows_here * (D / 4); x += 64 * W) {
        const int r = x / (D / 4), d = 4 * (x % (D / 4));
        float mm = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < W; ++i) mm = fmaxf(mm, lds.m[i][r]);
        const float mb = mm == -__builtin_inff() ? 0.f : mm;
        float ll = 0.f;
        float4_t oo = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int i = 0; i < W; ++i) {
            const float f = __builtin_amdgcn_exp2f(lds.m[i][r] - mb);
            ll = __builtin_fmaf(f, lds.l[i][r], ll);
            const float4_t t = *reinterpret_cast<const float4_t *>(&lds.o[i][r][d]);
#pragma unroll
            for (int c = 0; c < 4; ++c) oo[c] = __builtin_fmaf(f, t[c], oo[c]);
        }
        const int tr = a.group.div((uint32_t)(r0 + r));
        store_row<CT, D>(a, nsplit, a.splits_p + split, tok0 + tr, kvh * grp + r0 + r - tr * grp, d, oo, mm, ll);
    }
}

// The shared prefix: waves take different rows of the same tiles.
template <typename CT, int D, int RT, bool P16>
__device__ __forceinline__ void prefix_part(const AttnShared &a, AttnLds<D, true> &lds, int id, int tid) {
    using Lds = AttnLds<D, true>;
    constexpr int W = kAttnWaves;
    constexpr int RI = 512 / D;              // rows of a 1 KiB load
    constexpr int LR = D / 8;                // 16-byte pieces of a row
    constexpr int NK = kAttnTile / RI;       // loads for a tile's keys, and as many for its values
    constexpr int NI = 2 * NK / W;           // loads of a wave per tile
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), j = lane & 15, g = lane >> 4;
    const int x = a.xcd_p ? id & 7 : 0, id8 = a.xcd_p ? id >> 3 : id;
    const int y = a.groups_p.div((uint32_t)id8), rg = id8 - y * (int)a.groups_p.d;
    const int u = a.xcd_p ? y * 8 + x : y;
    const int split = a.heads.div((uint32_t)u), kvh = u - split * a.n_kv;
    const int r0 = (rg * W + wave) * RT * 16;

    Rows<CT, D, RT> w;
    w.init(a, r0, a.rows_p, 0, kvh, 0, a.prefix_len, j, g);
    const int ntile = (a.prefix_len + kAttnTile - 1) / kAttnTile;
    const int per = a.div_p.div((uint32_t)(ntile + a.splits_p - 1));
    const int ta = min(ntile, per * split), tb = min(ntile, per * (split + 1));
    // the first tile some wave's rows see differently (to the end: theirs alone)
    if (lane == 0) lds.least[wave] = w.lim_lo < w.lim_hi ? w.lim_lo / kAttnTile : tb, lds.most[wave] = w.lim_hi;
    __syncthreads();
    int t_split = tb, t_last = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) t_split = min(t_split, lds.least[i]), t_last = max(t_last, lds.most[i]);
    t_split = __builtin_amdgcn_readfirstlane(max(ta, t_split));
    t_last = __builtin_amdgcn_readfirstlane(min(tb, (t_last + kAttnTile - 1) / kAttnTile));

    KeyTile<CT, D, P16> kt{a, a.table, static_cast<const uint8_t *>(a.kc) + 2 * (int64_t)kvh * a.head_stride,
                           static_cast<const uint8_t *>(a.vc) + 2 * (int64_t)kvh * a.head_stride, lds.row[wave], {0, 0}};
    // This wave's share of a tile's loads: loads q = wave NI .. + NI, of which load q covers rows RI (q % NK) ..
    // of the keys (q < NK) or values; all lie in one half of the tile.  Lane l takes the 16 bytes whose place
    // in the load's kilobyte is l: of the keys piece l % LR of row l / LR, swizzled by the row; of the values
    // [16 dims][row][half of them], so that a transposing read finds 16 dims of 4 rows in 128 bytes.
    const auto swizzle = [](int row) { return (D == 64 ? row >> 1 : row) & (LR < 16 ? LR - 1 : 15); };
    const bool my_keys = wave * NI < NK;
    const int row0 = wave * NI % NK * RI;
    const uint32_t my_step = my_keys ? 1024u : (uint32_t)Lds::kBlock, my_ring = my_keys ? Lds::kTileBytes : Lds::kValueBytes;
    const uint32_t my_lds = (my_keys ? (uint32_t)(uintptr_t)&lds.ring.k[0][0] : (uint32_t)(uintptr_t)&lds.ring.v[0][0]) +
                            (uint32_t)(row0 / RI) * my_step;
    const uint8_t *my_base = my_keys ? kt.kbase : kt.vbase;
    const int in_row = my_keys ? lane / LR : D == 64 ? (lane >> 3 & 1) * 4 + (lane >> 1 & 3) : lane >> 1 & (RI - 1);
    const auto piece = [&](int i) {
        return 16 * (my_keys ? (lane % LR) ^ swizzle(row0 + i * RI + in_row) : 2 * (lane / (D == 64 ? 16 : 2 * RI)) + (lane & 1));
    };
    // The next tile to load (P16): this wave's half's index in the table, place in the page, page number (read
    // a tile ahead) and address.  What lies past the prefix takes its last page (and is masked).  Where a page
    // does not exist, NaN stands for its rows.
    int pi = 0, off = 0, page = 0;
    bool fresh = true;                       // (a new page: the address is still to be worked out)
    const uint8_t *src = nullptr;
    uint32_t voff[NI];
    const int last_pi = a.page.div((uint32_t)(a.prefix_len - 1)), psz = (int)a.page.d;
    if constexpr (P16) {
        const int key = ta * kAttnTile + (row0 & 16);
        pi = a.page.div((uint32_t)key);
        off = key - pi * psz;
        page = table_at(a.table, min(pi, last_pi));
#pragma unroll
        for (int i = 0; i < NI; ++i)
            voff[i] = (uint32_t)(2 * (((row0 & 15) + i * RI + in_row) * (int)a.token_stride) + piece(i));
    }
    int next = ta;
    const auto issue = [&](int buf) {
        const uint32_t dst = my_lds + (uint32_t)buf * my_ring;
        if constexpr (P16) {
            const bool ok = (uint32_t)page < (uint32_t)a.n_pages;
            if (fresh) src = my_base + 2 * ((int64_t)(ok ? page : 0) * a.page_stride + (int64_t)off * a.token_stride);
            if (ok) {
#pragma unroll
                for (int i = 0; i < NI; i += 2) lds_dma16x2(src, voff[i], voff[i + 1], dst + i * my_step, my_step);
            } else {
#pragma unroll
                for (int i = 0; i < NI; i += 2) lds_dma16x2(kNanRow, 0, 0, dst + i * my_step, my_step);
            }
            off += kAttnTile;
            src += 2 * kAttnTile * (int)a.token_stride;
            fresh = off >= psz;
            if (fresh) {
                off -= psz, ++pi;
                if (off >= psz) off -= psz, ++pi;    // (a page has 16 places at least)
                page = table_at(a.table, min(pi, last_pi));
            }
        } else {
            const uint32_t bad = kt.find(next * kAttnTile, 0, a.prefix_len, lane);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int row = row0 + i * RI + in_row;
                const uint8_t *p = my_base + kt.row(row) + piece(i);
                lds_dma16((bad >> row) & 1u ? reinterpret_cast<const uint8_t *>(kNanRow) : p, dst + i * my_step);
            }
        }
        ++next;
    };
    // A tile's keys are needed a tile earlier than its values: its scores are worked out beside the softmax
    // of the tile before.  So the waves that load keys are three tiles ahead, the others two.
    const int ahead = my_keys ? 3 : 2;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < ahead && next < t_split) issue(i);
    const auto load_k = [&](int buf) {
        const uint8_t *kb = lds.ring.k[buf];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < D / 32; ++s)
                w.k[h][s] = *reinterpret_cast<const u32x4_t *>(kb + (16 * h + j) * 2 * D + 16 * ((4 * s + g) ^ swizzle(16 * h + j)));
    };
    // the values' operands: of 16 dims 16 e .. and 4 keys each, read transposed
    u32x4_t va[D / 16];
    const int v_at = D == 64    ? (g >> 1) * Lds::kBlock + (g & 1) * 128 + 8 * j
                     : D == 128 ? g * Lds::kBlock + 8 * j
                                : (2 * g + (j >> 3)) * Lds::kBlock + 8 * (j & 7);
    const auto load_v = [&](int buf) {
        const uint8_t *vb = lds.ring.v[buf] + v_at;
#pragma unroll
        for (int e = 0; e < D / 16; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x2_t r = read_transposed(vb + h * (16 / RI) * Lds::kBlock + e * (D == 64 ? 256 : 32 * RI));
                va[e][2 * h] = r.x, va[e][2 * h + 1] = r.y;
            }
    };
    float4_t sc[RT][2];
    if (ta < t_split) {
        if (my_keys && ta + 2 < t_split) wait_vmcnt<2 * NI>();
        else wait_vmcnt<0>();
        __syncthreads();
        load_k(0);
#pragma unroll
        for (int t = 0; t < RT; ++t) w.scores(sc[t], t);
        settle();
    }
    int buf = 0;
    for (int tile = ta; tile < t_split; ++tile) {
        const int buf1 = buf == 2 ? 0 : buf + 1, buf2 = buf == 0 ? 2 : buf - 1;
        // this wave's share of this tile's values (the next tile's keys) is here, its next NI loads may still be
        // on their way ...
        if (next > tile + ahead - 1) wait_vmcnt<NI>();
        else wait_vmcnt<0>();
        __syncthreads();                     // ... and everyone's; and what was here before is read
        const int key0 = tile * kAttnTile;
        const bool work = w.lim_hi > key0;
        if (next < t_split) issue(my_keys ? buf : buf2);
        if (work) {
            load_k(buf1);                    // (past the last tile: not used)
            load_v(buf);
            const bool edge = key0 + kAttnTile > w.lim_hi;
            Weights p[RT];
            if (edge) {
#pragma unroll
                for (int t = 0; t < RT; ++t) w.mask(sc[t], t, key0, 0, 0, g);
                const u32x4_t keep = w.keys_kept(key0, 0, w.lim_hi, g);
#pragma unroll
                for (int e = 0; e < D / 16; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) va[e][i] &= keep[i];
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) w.raise(sc[t], t, a.scale2);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                p[t] = w.weights(sc[t], t, a.scale2);
                w.scores(sc[t], t);          // of the next tile
            }
            w.values(p, va);
        }
        buf = buf1;
    }
    for (int tile = t_split; tile < t_last; ++tile) {
        const int key0 = tile * kAttnTile;
        __syncthreads();
        issue(0);
        wait_vmcnt<0>();
        __syncthreads();
        if (w.lim_hi > key0) {
            load_k(0);
            load_v(0);
#pragma unroll
            for (int t = 0; t < RT; ++t) w.mixed_tile(t, a.scale2, key0, 0, 0, g, [&](int e) { return va[e]; });
        }
    }
    __syncthreads();                         // (the tile buffers become O areas)
    float *area = &lds.o[wave][0][0];
    w.finish(0);
    const int grp = (int)a.group.d, nsplit = a.splits_p + (a.wgs_o ? (int)a.splits_o.d : 0);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        w.template o_to_lds<true>(area, t, j, g);
        if (g == 0) lds.m[wave][j] = w.m[t], lds.l[wave][j] = w.l[t][0];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int rows_here = min(a.rows_p - r0 - 16 * t, 16);
#pragma unroll 1
        for (int i = lane; i < rows_here * (D / 4); i += 64) {
            const int r = i / (D / 4), d = 4 * (i % (D / 4)), rr = r0 + 16 * t + r;
            const int tok = a.group.div((uint32_t)rr);
            store_row<CT, D>(a, nsplit, split, tok, kvh * grp + rr - tok * grp, d,
                             *reinterpret_cast<const float4_t *>(area + r * (D + 4) + d), lds.m[wave][r], lds.l[wave][r]);
        }
    }
}

// RTP: 16-row tiles of a wave in the prefix part; 0: there is none.
// Measured with 32 query and 8 key heads of 128, bfloat16, in a graph: one sequence of 777 keys 11.5 us (3.2 MB:
// latency of seven dependent tiles); of 100000 76.5 us (410 MB, 5.4 TB/s); 16 sequences over 4096 shared keys
// and up to 513 own 16.5 us with the join (36 MB); 64 over 32768 and up to 1025 87 us (270 MB, 3.1 TB/s: a
// prefix tile takes 1.1 us where HBM would need 0.35, and the splits' results are written and read back,
// 2 x 17 MB).
template <typename CT, int D, int RTP, bool P16>
__global__ __launch_bounds__(64 * kAttnWaves, D == 256 ? 1 : 2) void attn_rows(AttnShared a) {
    __shared__ AttnLds<D, (RTP > 0)> lds;
    if constexpr (RTP > 0) {
        if ((int)blockIdx.x < a.wgs_p) {
            prefix_part<CT, D, RTP, P16>(a, lds, blockIdx.x, threadIdx.x);
            return;
        }
    }
    own_part<CT, D, (RTP > 0), P16>(a, lds, (int)blockIdx.x - a.wgs_p, threadIdx.x);
}

// Joins the splits (at most 64) of a row: a workgroup per row, D/4 lanes for a split's O, so that a row's
// loads go out together.  2048 rows of 17 splits of 128 (18 MB) 6.0 us, 512 rows 3.9: the launch and two
// dependent loads.
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

AttnPlan attn_plan(int64_t n_seqs, int64_t n_q, int64_t n_kv, int64_t dim, int64_t n_qt, int64_t prefix_len,
                   int64_t max_len) {
    AttnPlan p{};
    const int64_t rows_o = n_qt * (n_q / n_kv), rows_p = n_seqs * rows_o;
    const auto tiles = [](int64_t keys) { return (keys + kAttnTile - 1) / kAttnTile; };
    const auto div_up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
    const auto splits = [&](int64_t want, int64_t most) {
        const int64_t s = want < most ? want : most;
        return s < 1 ? (int64_t)1 : s > kAttnMaxSplits ? (int64_t)kAttnMaxSplits : s;
    };
    p.groups_o = div_up(rows_o, 16);
    // The prefix has a part of its own unless it is of one sequence with one tile of rows, or all is
    // short and few: then a sequence's workgroups take all of its keys, prefix included (read once per
    // sequence, from the L2).  In us, so and with a part of its own: 8 sequences of 4 query tokens and 2 key
    // heads with 1300 keys 9.5 and 10.4, with 1750 10.3 and 10.9; 8 sequences of 8 key heads with 1000 keys
    // 9.7 and 10.8, with 1300 12.5 and 11.0, with 1600 12.8 and 11.0; 16 of them with 1200 keys 15.7 and 12.4.
    const int64_t wgs = n_seqs * n_kv * p.groups_o;
    p.joint = prefix_len > 0 && ((n_seqs == 1 && rows_p <= 16) || (tiles(max_len) <= 56 && tiles(max_len) * wgs <= 2304));
    const bool shared = prefix_len > 0 && !p.joint;
    if (shared) {
        // Row tiles of a wave (2 read the tiles from LDS half as often, 1 gives twice the workgroups; 256 dims
        // have registers for 1) and the number of splits weigh the tiles of a split, by a workgroup alone on its CU or
        // beside another, against the splits' results, written and read back.  The weights are not times: they were
        // fitted, at 128 dims, and the choice they make is what was measured.  With 8 key heads of 32 query heads, in us,
        // row tiles / splits: 64 sequences of 128 dims over 32768 keys choose 2/16, 90 (2/24 85, 2/32 97, 1/12 95), over
        // 8192 1/8, 50 (2/12 49, 2/16 50), over 131072 2/32, 235 (2/24 246, 1/16 280); 16 over 4096 1/16, 17.3 (1/8 22,
        // 1/32 19); of 64 dims over 32768 2/32, 53 (1/24 55), over 8192 29 (2/16 27).  256 dims, of which a CU
        // holds one workgroup, fit less well: 64 sequences over 8192 keys 114 (1/4 102), over 32768 231 (1/12 226), 16 over
        // 4096 30 (1/16 26).  At least four tiles each.
        constexpr double alone[2] = {0.55, 0.75}, beside[2] = {0.98, 1.15};
        const int64_t t = tiles(prefix_len), part = rows_p * n_kv * dim * 4;
        double best = 0;
        for (int rt = 1; rt <= (dim < 256 && rows_p > 16 * kAttnWaves ? 2 : 1); ++rt) {
            const int64_t groups = div_up(rows_p, 16 * kAttnWaves * rt), units = groups * n_kv;
            for (int64_t n = 1; n <= kAttnMaxSplits && (n == 1 || 4 * n <= t); ++n) {
                const double tile = n * units <= 256 ? alone[rt - 1] : beside[rt - 1] * (double)div_up(n * units, 512);
                const double us = (double)div_up(t, n) * tile + (double)(n * part) / 0.75e6;
                if (p.splits_p == 0 || us < best) best = us, p.splits_p = n, p.row_tiles = rt, p.groups_p = groups;
            }
        }
    }
    const int64_t own = shared ? tiles(max_len) - prefix_len / kAttnTile : tiles(max_len);
    // own keys: a few tiles a wave are taken at once; beyond, enough workgroups for the chip, two tiles a wave at
    // least.  A split saves the GPU's time and costs a caller that is not captured in a graph a second launch, some 4 us
    // of its own.  With 8 key heads of 128, in us, GPU / back to back from Python: one sequence of 640 keys in one split
    // 9.3 / 11.2, in 3 8.5 / 15.6; 777 11.5 / 11.8 and 9.6 / 15.7; 896 11.4 / 11.8 and 9.7 / 15.7; 1000 12.7 / 13.0
    // and in 4 8.9 / 15.7; 1200 14.9 / 15.1 and 9.7 / 15.4.  At 28 tiles the one form stops costing the GPU less than
    // the other costs the caller.  16 sequences: 1000 keys 15.8 / 15.6 in one, 16.5 / 16.6 in 4; 1280 20.4 / 20.2 and
    // 19.5 / 19.4.
    const int64_t few = shared ? 20 : wgs >= 128 ? 40 : 28;
    if (!shared || max_len > prefix_len)
        p.splits_o = own <= few ? 1 : splits(div_up(512, wgs), own / (2 * kAttnWaves));
    const int64_t n = p.splits_p + p.splits_o;
    const int64_t rows_wgs = n_kv * (p.groups_p * p.splits_p + p.groups_o * p.splits_o * n_seqs), out_rows = rows_p * n_kv;
    p.groups = n > 1 && out_rows > rows_wgs ? out_rows : rows_wgs;      // (attn_rows, attn_join)
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
    a.own_from = p.splits_p ? a.prefix_len : 0;
    a.joint_len = p.joint && a.n_seqs > 1 ? a.prefix_len : 0;   // (one sequence: row 0 is its own)
    const int64_t units_p = a.n_kv * p.splits_p;
    a.xcd_p = p.groups_p > 1 && units_p % 8 == 0;
    a.wgs_p = (int)(p.groups_p * units_p);
    a.wgs_o = (int)(p.groups_o * a.n_kv * p.splits_o * a.n_seqs);
    const int64_t n_out = (int64_t)a.rows_p * a.n_kv;
    const int nsplit = (int)(p.splits_p + p.splits_o);
    a.part_ml = a.part_o + nsplit * n_out * dim;
    const dim3 grid((unsigned)(a.wgs_p + a.wgs_o));
    const bool p16 = a.page.d % 16 == 0 && a.joint_len % 16 == 0;
    auto run = [&](auto ctag, auto d, auto rtp) -> hipError_t {
        using CT = decltype(ctag);
        constexpr int D = decltype(d)::value, RTP = decltype(rtp)::value, T = 64 * kAttnWaves;
        if (p16) attn_rows<CT, D, RTP, true><<<grid, T, 0, s>>>(a);
        else attn_rows<CT, D, RTP, false><<<grid, T, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || nsplit == 1) return e;
        attn_join<CT, D><<<dim3((unsigned)n_out), 256, 0, s>>>(a, nsplit);
        return hipGetLastError();
    };
    auto by_rows = [&](auto ctag, auto d) -> hipError_t {
        constexpr int big = decltype(d)::value == 256 ? 1 : 2;
        if (p.row_tiles == 0) return run(ctag, d, std::integral_constant<int, 0>{});
        if (p.row_tiles == 1) return run(ctag, d, std::integral_constant<int, 1>{});
        return run(ctag, d, std::integral_constant<int, big>{});
    };
    auto by_dim = [&](auto ctag) -> hipError_t {
        if (dim == 64) return by_rows(ctag, std::integral_constant<int, 64>{});
        if (dim == 128) return by_rows(ctag, std::integral_constant<int, 128>{});
        return by_rows(ctag, std::integral_constant<int, 256>{});
    };
    return ct == Act::F16 ? by_dim(_Float16{}) : by_dim(bf16_t{});
}

}  // namespace q2_0
