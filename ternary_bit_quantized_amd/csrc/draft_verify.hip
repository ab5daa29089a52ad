// Verification of drafted tokens, and the token that follows the accepted ones.
//
// With p = softmax(target / T) and q = softmax(draft / T) of a drafted place, its token t is taken where
// u q(t) < p(t); at the first that is not, the token comes from max(p - q, 0), and after the last from p
// itself, both by the inverse of the running sum at a given number.  Every output is a whole number
// that hangs on a comparison of sums over the vocabulary, so exponentials and sums are in 64 bits: in 32
// a running sum over 10^5 tokens is off by some 10^-7 of the whole, which moves about one choice in a
// thousand to the token beside it.
//
//   draft_stats  one pass over every row that may be needed: maximum and sum of exponentials of each chunk
//                (a running maximum in registers, rescaled where a pass raises it)
//   draft_sums   each workgroup joins its sequence's chunks, decides how many drafts are taken, and sums
//                max(p - q, 0) of the deciding row over tiles of 512 tokens; the last workgroup of a sequence
//                finds the tile, then the token, at which the running sum passes the number
//
// Given probabilities need no statistics, and find the token in a launch of its own (draft_pick).  All sums are in a fixed
// order: results are the same in every run.
//
// What bounds it, in a graph.  64 sequences of 4 drafts over 151936 f32 logits, 350 MB: 84 to 91 us.  57 to 62 of them are the
// statistics, by counters: the vector units are busy for 37 of 57 us (14 64-bit instructions an exponential, 22.6 million of
// all kinds on 1024 SIMDs), with 4.2 waves a SIMD on average, which spend 44 % of their time waiting to issue and 35 %
// at waits (their loads alone take 43 us: 6.5 TB/s for the 283 MB that are needed).  29 to 31 are the tile sums (deciding 7.6,
// two rows' exponentials 11, the token 3).  The same logits in bfloat16: 88 us, since the instructions are the same (the
// statistics 53) and the tile sums' waves (39) are at waits 2.4 times as long.  One sequence of f32: 15.4 us, two launches of
// dependent steps: deciding 4, a tile 1.8, the token 3.  16 sequences of 5 found drafts over 50001 bfloat16 logits 18.5 us; 32
// of 3 given probabilities over 32003, 8.0 us.  (The statistics' loads are non-temporal: 64 sequences took 76.7 us a pass with
// other work between, 80.5 with plain ones.)
#include "serve_common.h"

namespace q2_0 {

constexpr int kMaxRows = 2 * Q2_0_DRAFT_MAX + 1;
constexpr int kTile = 512;            // tokens of a tile sum (of 1024: one chat 1.6 us more, 64 sequences 1.3 less)
constexpr int kCountEvery = 32;       // counters of sequences in lines of their own: side by side 400 workgroups wait 2 us for 16
constexpr int kPass = 4096;           // values of a workgroup's pass: 16 a thread

// 2^r for r in [-1/2, 1/2]: the polynomial of degree 9 that meets it at the Chebyshev points (relative error 1.9e-14, below
// 2^-45).  Of degree 8 the error is 1.1e-12 and 64 sequences of 4 drafts take 80.3 us a pass in place of 83.2, but 21 of
// 6 million two-token rows, whose number is the float32 next to their probability, are decided otherwise than they are defined.
__device__ __forceinline__ double exp2_frac(double r) {
    double e = 1.020590550210069e-07;
    e = fma(e, r, 1.3259645241948732e-06);
    e = fma(e, r, 1.5252672924257465e-05);
    e = fma(e, r, 0.0001540343375126647);
    e = fma(e, r, 0.0013333558200796013);
    e = fma(e, r, 0.00961812919393429);
    e = fma(e, r, 0.05550410866465166);
    e = fma(e, r, 0.2402265069564034);
    e = fma(e, r, 0.6931471805599462);
    return fma(e, r, 1.0000000000000135);
}

constexpr double kBig = 6755399441055744.0;      // 1.5 2^52: x + kBig is x rounded to a whole number, in the low bits

// 2^y for y <= 0, 0 below -1100 and for NaN.
__device__ __forceinline__ double exp2_64(double y) {
    y = fmax(y, -1100.0);
    const double t = y + kBig;
    return __builtin_amdgcn_ldexp(exp2_frac(y - (t - kBig)), (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
}

// The exponentials of a row (or a part of one) of largest value m: 2^(k x - ref) with ref the whole number next to k m.  ref goes
// into the exponent: with t = k x + (kBig - ref), one rounding to a whole number, q = t - (kBig - ref) and r = k x - q, a value
// takes 14 64-bit instructions, and k x is not rounded before its whole part is gone.
// Where k m is 2^28 and more, float32 has no value 1000 below m in the exponent to stop at (`low` is off by 16 there): x - m takes
// the place of x (`off`; else 0) with ref 0.  The difference is exact in float32 for x within a factor of 2 of m, and the
// others are 2^-2^27 and less.
struct RowExps {
    double big;            // kBig - ref
    float off, low;        // values below `low`, 2^-1000 of the largest, count nothing
    // for sums: 2^-1000 and less count as that; x less `off` already
    __device__ __forceinline__ double of(float x, double k) const {
        const double v = (double)__builtin_elementwise_maximum(x, low);      // (NaN stays; fmaxf would take two instructions)
        const double t = fma(v, k, big);
        u32x2_t e = __builtin_bit_cast(u32x2_t, exp2_frac(fma(v, k, -(t - big))));
        e.y += (uint32_t)__builtin_bit_cast(uint64_t, t) << 20;
        return __builtin_bit_cast(double, e);
    }
    __device__ __forceinline__ double exact(float x, double k) const {
        const double v = of(x - off, k);
        return x - off < low ? 0.0 : v;
    }
};
struct Exps : RowExps {
    double k;
    float m, d;            // d: 1000 / k
    __device__ __forceinline__ void scale(double by) { k = by, d = 1000.f / (float)by; }
    __device__ __forceinline__ void about(float top) {
        const double mk = (double)top * k;
        const bool whole = fabs(mk) < 0x1p28;
        m = top;
        off = whole ? 0.f : top;
        big = kBig - (whole ? rint(mk) : 0.0);
        low = (whole ? top : 0.f) - d;
    }
    // A sum about this part's reference as one about the whole's (all.m >= m): the whole number where `off` is 0, else k m
    // itself.  Where they are of two kinds, the product and the whole number are subtracted in one rounding (of a product of
    // 2^28 alone it would be 2^-25).
    __device__ __forceinline__ double share_of(double z, const Exps &all) const {
        if (off == 0.f && all.off == 0.f) return __builtin_amdgcn_ldexp(z, (int)fmax(all.big - big, -4000.0));
        const double lower = off == 0.f         ? -fma((double)all.m, k, big - kBig)
                             : all.off == 0.f ? fma((double)m, k, all.big - kBig)
                                              : ((double)m - (double)all.m) * k;
        return z * exp2_64(lower);
    }
};

__device__ __forceinline__ double nan64() { return __builtin_nan(""); }

__device__ __forceinline__ float wave_max(float v) {
    const float none = -__builtin_inff();
    v = fmaxf(v, lane_move<0x111, 0xf>(v, none));
    v = fmaxf(v, lane_move<0x112, 0xf>(v, none));
    v = fmaxf(v, lane_move<0x114, 0xf>(v, none));
    v = fmaxf(v, lane_move<0x118, 0xf>(v, none));
    v = fmaxf(v, lane_move<0x142, 0xa>(v, none));
    v = fmaxf(v, lane_move<0x143, 0xc>(v, none));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// log2(e) / temperature, which counts as at most 2^100 and at least 2^-100 (logits would be out of all proportion to it); NaN
// for one that is not positive.
__device__ __forceinline__ double scale_of(const DraftVerify &a, int s) {
    if (!a.temperature) return 1.4426950408889634074;
    const float t = a.temperature[s];
    return t > 0.f ? 1.4426950408889634074 / (double)fmaxf(fminf(t, 0x1p100f), 0x1p-100f) : nan64();
}

__device__ __forceinline__ bool greedy_of(const DraftVerify &a, int s) { return a.temperature && a.temperature[s] == 0.f; }

// The largest of three, NaN if one is: one instruction that finds both.
__device__ __forceinline__ float max3(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

template <typename XT>
struct Vec {                          // 16 bytes of a row
    static constexpr int n = 16 / sizeof(XT);
    static constexpr int each = kPass / 256 / n, pass = kPass / n;   // vectors of a thread and of a pass
    float x[n];
};

__device__ __forceinline__ void unpack(u32x4_t v, Vec<float> &o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = v[i];      // (a cast of the element itself would read the vector's first)
        o.x[i] = __builtin_bit_cast(float, b);
    }
}
__device__ __forceinline__ void unpack(u32x4_t v, Vec<_Float16> &o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = v[i];
        const half2_t h = __builtin_bit_cast(half2_t, b);
        o.x[2 * i] = (float)h.x, o.x[2 * i + 1] = (float)h.y;
    }
}
__device__ __forceinline__ void unpack(u32x4_t v, Vec<bf16_t> &o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.x[2 * i] = __builtin_bit_cast(float, v[i] << 16);
        o.x[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
    }
}

// A thread's vectors of the pass that begins at vector v of a row whose first element is `shift` elements past a 16-byte
// boundary; what is outside the row (or at `end` and after it) is -inf and not read.
template <typename XT>
__device__ __forceinline__ void load_pass(const XT *row, int shift, int n_vocab, int v, int end, Vec<XT> (&x)[Vec<XT>::each]) {
    constexpr int VE = Vec<XT>::n;
    const int first = v * VE - shift;
    if (first >= 0 && v + Vec<XT>::pass <= end && first + kPass <= n_vocab) {
#pragma unroll
        for (int i = 0; i < Vec<XT>::each; ++i)
            unpack(__builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(row + first + (i * 256 + (int)threadIdx.x) * VE)), x[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < Vec<XT>::each; ++i) {
        const int w = v + i * 256 + (int)threadIdx.x, e = w * VE - shift;
        if (w < end && e >= 0 && e + VE <= n_vocab) {
            unpack(*reinterpret_cast<const u32x4_t *>(row + e), x[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                x[i].x[j] = w < end && e + j >= 0 && e + j < n_vocab ? act_to_f32(row[e + j]) : -__builtin_inff();
        }
    }
}

template <typename XT>
__global__ __launch_bounds__(256) void draft_stats(DraftVerify a, DraftPlan p) {
    const int b = (int)(blockIdx.x / (unsigned)p.chunks), c = (int)(blockIdx.x % (unsigned)p.chunks);
    const int per = a.max_draft + 1, n_target = a.n_seqs * per;
    const bool is_draft = b >= n_target;
    const int s = is_draft ? (b - n_target) / a.max_draft : b / per;
    const int j = is_draft ? (b - n_target) % a.max_draft : b % per;
    if (!is_draft && j == 0 && c == 0 && threadIdx.x == 0) reinterpret_cast<int *>(a.ws + p.off_done)[s * kCountEvery] = 0;
    const int nd = a.n_draft[s];
    if (nd < 0 || nd > a.max_draft || j >= nd + (is_draft ? 0 : 1)) return;
    const bool greedy = greedy_of(a, s);
    if (greedy && is_draft) return;
    const XT *row = is_draft ? static_cast<const XT *>(a.draft) + (int64_t)(b - n_target) * a.ld_draft
                             : static_cast<const XT *>(a.target) + (int64_t)b * a.ld_target;
    constexpr int VE = Vec<XT>::n;
    const int shift = (int)(((uintptr_t)row & 15) / sizeof(XT));
    const int nv = (a.n_vocab + shift + VE - 1) / VE;
    const int v0 = c * p.chunk_vecs, v1 = nv < v0 + p.chunk_vecs ? nv : v0 + p.chunk_vecs;
    float m = -__builtin_inff();
    double z = 0.0;
    int arg = 0x7fffffff;
    bool bad = false;
    Exps ex;
    ex.scale(scale_of(a, s));
    for (int v = v0; v < v1; v += Vec<XT>::pass) {
        Vec<XT> x[Vec<XT>::each];
        load_pass(row, shift, a.n_vocab, v, v1, x);
        float top = m;
#pragma unroll
        for (int i = 0; i < Vec<XT>::each; ++i)
#pragma unroll
            for (int e = 0; e < VE; e += 2) top = max3(top, x[i].x[e], x[i].x[e + 1]);
        bad |= top != top;
        if (greedy) {
            if (top > m) {
                m = top;
#pragma unroll
                for (int i = Vec<XT>::each - 1; i >= 0; --i)
#pragma unroll
                    for (int e = VE - 1; e >= 0; --e)
                        if (x[i].x[e] == top) arg = (v + i * 256 + (int)threadIdx.x) * VE - shift + e;
            }
            continue;
        }
        if (top > m) {
            const Exps before = ex;
            ex.about(top);
            z = m == -__builtin_inff() ? 0.0 : before.share_of(z, ex);
            m = top;
        }
        if (m == -__builtin_inff()) continue;
        if (ex.off == 0.f) {
#pragma unroll
            for (int i = 0; i < Vec<XT>::each; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) z += ex.of(x[i].x[e], ex.k);
        } else {
#pragma unroll
            for (int i = 0; i < Vec<XT>::each; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) z += ex.of(x[i].x[e] - ex.off, ex.k);
        }
    }
    __shared__ float wm[4];
    __shared__ double wz[4];
    __shared__ int warg[4], wbad[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float top = wave_max(m);
    if (lane == 0) wm[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
    if (greedy) {
        int at = m == top ? arg : 0x7fffffff;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const int o = __shfl_xor(at, off);
            at = o < at ? o : at;
        }
        if (lane == 0) warg[wave] = at;
    } else {
        const Exps mine = ex;
        ex.about(top);
        z = m == -__builtin_inff() ? 0.0 : mine.share_of(z, ex);
        z = wave_sum(z);
    }
    const bool any = __ballot(bad) != 0;
    if (lane == 0) wz[wave] = z, wbad[wave] = any;
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool none = wbad[0] | wbad[1] | wbad[2] | wbad[3] || top == __builtin_inff();
        const double sum = greedy ? 1.0 : ((wz[0] + wz[1]) + wz[2]) + wz[3];
        reinterpret_cast<double *>(a.ws + p.off_z)[blockIdx.x] = none ? nan64() : top == -__builtin_inff() ? 0.0 : sum;
        reinterpret_cast<float *>(a.ws + p.off_max)[blockIdx.x] = top;
        if (greedy) {
            int at = 0x7fffffff;
            for (int w = 0; w < 4; ++w) at = warg[w] < at ? warg[w] : at;
            reinterpret_cast<int *>(a.ws + p.off_arg)[blockIdx.x] = at;
        }
    }
}

// What decides a sequence's next token.
struct Pick {
    RowExps p, q;
    double k, inv_p, inv_q;               // p(x) = p.exact(x, k) inv_p
    int64_t row_p, row_q;                 // rows of target and draft
    int taken;                            // drafts taken; < 0: the sequence is left out
    int kind;                             // kFixed: `token`; else what is taken from p
    int token;                            // the next token (kFixed), the token to leave out (kOneHot); kUnseen: of a given draft
                                          // row nothing above 0 has been read
};
enum { kFixed = 0, kPlain = 1, kOneHot = 2, kMinus = 3 };
constexpr int kUnseen = -2;

// (given probabilities below 0 count as 0; NaN stays)
template <bool PROBS>
__device__ __forceinline__ double prob(float x, const RowExps &e, double k, double inv) {
    return PROBS ? (double)(x < 0.f ? 0.f : x) : e.exact(x, k) * inv;
}

// All threads of the workgroup; the result is in `pick` after a barrier.
template <typename XT, bool PROBS>
__device__ void decide(const DraftVerify &a, const DraftPlan &p, int s, Pick &pick) {
    __shared__ RowExps most[kMaxRows];
    __shared__ double whole[kMaxRows];           // sums of exponentials
    __shared__ int arg[kMaxRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = a.max_draft + 1;
    const double *all_z = reinterpret_cast<const double *>(a.ws + p.off_z);
    const float *all_m = reinterpret_cast<const float *>(a.ws + p.off_max);
    const int *all_at = reinterpret_cast<const int *>(a.ws + p.off_arg);
    // Rows of the target, then of the draft, whether they are needed or not: what their first four have is asked for together
    // with the number of drafts and the drafted tokens (what was not needed was not written, and is not used below).
    const int rows = PROBS ? 0 : per + (a.draft ? a.max_draft : 0);
    auto row_of = [&](int r) { return (r < per ? (int64_t)s * per + r : (int64_t)a.n_seqs * per + (int64_t)s * a.max_draft + (r - per)) * p.chunks; };
    float m[4];
    double z[4];
    int at[4];
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = row_of(r0 + 4 * i < rows ? r0 + 4 * i : r0) + (lane < p.chunks ? lane : 0);
            m[i] = all_m[c];
            z[i] = all_z[c];
            at[i] = a.temperature ? all_at[c] : 0x7fffffff;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane >= p.chunks) m[i] = -__builtin_inff(), z[i] = 0.0, at[i] = 0x7fffffff;
    };
    const int nd = a.n_draft[s];
    int tok = -1;
    float u = 0.f;
    const int64_t row_p = (int64_t)s * per + lane, row_q = (int64_t)s * a.max_draft + lane;
    if (wave == 0 && lane < a.max_draft) tok = a.tokens[row_q], u = a.u[row_p];
    if (wave < rows) load(wave);
    if (nd < 0 || nd > a.max_draft) {
        if (threadIdx.x == 0) pick.taken = -1, pick.kind = kFixed, pick.token = -1;
        return;
    }
    const bool greedy = !PROBS && greedy_of(a, s);
    const double k = PROBS ? 0.0 : scale_of(a, s);
    // the drafted tokens' values arrive while the rows are joined
    float xt = 0.f, xd = 0.f;
    const bool known = lane < nd && tok >= 0 && tok < a.n_vocab;
    if (known && !greedy) {
        xt = act_to_f32(static_cast<const XT *>(a.target)[row_p * a.ld_target + tok]);
        if (a.draft) xd = act_to_f32(static_cast<const XT *>(a.draft)[row_q * a.ld_draft + tok]);
    }
    if (!PROBS) {
        // four rows of a wave side by side: loads, maxima and sums of one wait for memory and for each other
        for (int r0 = wave; r0 < rows; r0 += 16) {
            if (r0 != wave) load(r0);
            float top[4];
            Exps part, all;
            part.scale(k), all.scale(k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t from = row_of(r0 + 4 * i < rows ? r0 + 4 * i : r0);
                for (int c = lane + 64; c < p.chunks; c += 64) {         // (rows of over 64 chunks)
                    const float om = all_m[from + c];
                    const double oz = all_z[from + c];
                    if (greedy) {
                        z[i] += oz;
                        if (om > m[i]) at[i] = all_at[from + c];         // (chunks of a lane go up: the first of equals stays)
                        m[i] = fmaxf(m[i], om);
                    } else {
                        const float most = fmaxf(m[i], om);
                        all.about(most);
                        part.about(m[i]);
                        if (m[i] > -__builtin_inff()) z[i] = part.share_of(z[i], all);
                        part.about(om);
                        z[i] += om > -__builtin_inff() ? part.share_of(oz, all) : oz;
                        m[i] = most;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = wave_max(m[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all.about(top[i]);
                part.about(m[i]);
                // (a chunk of NaN: its sum is NaN and stays so)
                if (!greedy && m[i] > -__builtin_inff()) z[i] = part.share_of(z[i], all);
                at[i] = m[i] == top[i] ? at[i] : 0x7fffffff;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = wave_sum(z[i]);
            if (greedy)
#pragma unroll
                for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int o = __shfl_xor(at[i], off);
                        at[i] = o < at[i] ? o : at[i];
                    }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane == 0 && r0 + 4 * i < rows) {
                    all.about(top[i]);
                    most[r0 + 4 * i] = all;
                    whole[r0 + 4 * i] = z[i] > 0.0 && z[i] < __builtin_inf() ? z[i] : nan64();
                    arg[r0 + 4 * i] = z[i] == z[i] && top[i] > -__builtin_inff() ? at[i] : -1;
                }
        }
        __syncthreads();
    }
    if (wave != 0) return;
    bool yes = false;
    if (known) {
        if (greedy) {
            yes = arg[lane] == tok;
        } else {
            // u q < p, by the sums in place of their quotients
            const double pt = prob<PROBS>(xt, most[lane], k, 1.0), sp = PROBS ? 1.0 : whole[lane];
            const double qt = !a.draft ? 1.0 : prob<PROBS>(xd, most[per + lane], k, 1.0);
            const double sq = !a.draft || PROBS ? 1.0 : whole[per + lane];
            yes = (double)u * qt * sp < pt * sq && (!PROBS || pt < __builtin_inf());   // (given: of NaN neither comparison holds)
        }
    }
    const uint64_t no = __ballot(!yes);                  // (lanes from nd on: not taken)
    const int j = (int)__ffsll((unsigned long long)no) - 1;
    const int t = __builtin_amdgcn_readlane(tok, j);
    const bool seen = !PROBS || (__ballot(xd > 0.f) >> j & 1);
    if (lane == 0) {
        pick.taken = j;
        pick.k = k;
        pick.row_p = (int64_t)s * per + j;
        pick.row_q = (int64_t)s * a.max_draft + j;
        if (!PROBS) {
            pick.p = most[j], pick.inv_p = 1.0 / whole[j];
            if (j < nd && a.draft && !greedy) pick.q = most[per + j], pick.inv_q = 1.0 / whole[per + j];
        }
        if (greedy) pick.kind = kFixed, pick.token = arg[j];
        else if (j == nd) pick.kind = kPlain, pick.token = -1;
        else if (!a.draft) pick.kind = kOneHot, pick.token = t;
        else pick.kind = kMinus, pick.token = seen ? -1 : kUnseen;
    }
}

// The same values in scalar registers: a Pick comes from shared or global memory, the same for all lanes.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) { return __builtin_bit_cast(float, uniform(__builtin_bit_cast(int, v))); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}
__device__ __forceinline__ double uniform(double v) { return __builtin_bit_cast(double, uniform(__builtin_bit_cast(int64_t, v))); }
__device__ __forceinline__ RowExps uniform(const RowExps &e) { return RowExps{uniform(e.big), uniform(e.off), uniform(e.low)}; }
__device__ __forceinline__ Pick uniform(const Pick &v) {
    return Pick{uniform(v.p), uniform(v.q), uniform(v.k), uniform(v.inv_p), uniform(v.inv_q), uniform(v.row_p), uniform(v.row_q),
                uniform(v.taken), uniform(v.kind), uniform(v.token)};
}

// The values of N tokens from e on, `step` apart, for what is left of them.  Without branches (a place past the row
// reads its last token): with a branch around each the loads wait for one another.
template <int N, typename XT>
struct Tokens {
    float x[N], y[N];
    __device__ __forceinline__ void load(const DraftVerify &a, const Pick &pick, int kind, int e, int step) {
        const XT *t = static_cast<const XT *>(a.target) + pick.row_p * a.ld_target;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = e + i * step;
            x[i] = act_to_f32(t[at < a.n_vocab ? at : a.n_vocab - 1]);
        }
        if (kind == kMinus) {
            const XT *d = static_cast<const XT *>(a.draft) + pick.row_q * a.ld_draft;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = e + i * step;
                y[i] = act_to_f32(d[at < a.n_vocab ? at : a.n_vocab - 1]);
            }
        }
    }
    // token `at`, the i-th: not below zero, NaN where either is
    template <bool PROBS>
    __device__ __forceinline__ double left(const DraftVerify &a, const Pick &pick, int kind, int i, int at) const {
        double v = prob<PROBS>(x[i], pick.p, pick.k, pick.inv_p);
        if (kind == kMinus) v -= prob<PROBS>(y[i], pick.q, pick.k, pick.inv_q);
        if (PROBS && kind == kMinus && y[i] == __builtin_inff()) v = nan64();        // (p - inf would be nothing left)
        // (a given probability that is none stays one, of the token to leave out too)
        const bool out = at >= a.n_vocab || (kind == kOneHot && at == pick.token && !(PROBS && !(v < __builtin_inf())));
        return out || v <= 0.0 ? 0.0 : v;
    }
};

template <typename XT, bool PROBS>
__device__ __forceinline__ double tile_sum(const DraftVerify &a, const Pick &pick, int kind, int tile) {
    constexpr int N = kTile / 64;
    const int e = tile * kTile + (int)(threadIdx.x & 63);
    Tokens<N, XT> t;
    t.load(a, pick, kind, e, 64);
    double sum = 0.0;
    if (kind == kMinus) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            sum += t.template left<PROBS>(a, pick, kMinus, i, e + 64 * i);
            __builtin_amdgcn_sched_barrier(0);           // (side by side they take registers, and waves, away)
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) sum += t.template left<PROBS>(a, pick, kind == kOneHot ? kOneHot : kPlain, i, e + 64 * i);
    }
    return wave_sum(sum);
}

// Tile sums go from the workgroups that make them to the one that reads them by exchanges with memory alone, as their count
// does: written and read where all of the device's atomics meet, whatever the dies' caches hold.  A fence for the device
// instead would write back and drop a cache for every workgroup: 1280 of them took 155 us in place of 25.
__device__ __forceinline__ void put_sum(double *p, double v) {
    __hip_atomic_exchange(reinterpret_cast<uint64_t *>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double sum_of(double *p) {
    uint64_t none = 0;
    asm volatile("" : "+v"(none));       // (the compiler makes a load of an exchange that it sees to change nothing)
    return __builtin_bit_cast(double, __hip_atomic_fetch_or(reinterpret_cast<uint64_t *>(p), none, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}
// All threads: the workgroup's atomics have been performed.
__device__ __forceinline__ void sums_done() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// Running sums over the 256 threads in their order: the sum up to the thread itself; `total`: all.
__device__ __forceinline__ double run_256(double v, double *wave_sums, double &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = lanes_run(v);
    __syncthreads();                                     // (wave_sums may be read still)
    if (lane == 63) wave_sums[wave] = v;
    __syncthreads();
    const double s0 = wave_sums[0], s1 = wave_sums[1], s2 = wave_sums[2], s3 = wave_sums[3];
    total = ((s0 + s1) + s2) + s3;
    return v + (wave == 0 ? 0.0 : wave == 1 ? s0 : wave == 2 ? s0 + s1 : (s0 + s1) + s2);
}

// The first thread whose running sum is above r and that holds anything, else the last that does.
__device__ __forceinline__ int thread_at(double run, double own, double r, int *hits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t over = __ballot(own > 0.0 && run > r), some = __ballot(own > 0.0);
    if (lane == 0) {
        hits[wave] = over ? 64 * wave + (int)__ffsll((unsigned long long)over) - 1 : -1;
        hits[4 + wave] = some ? 64 * wave + 63 - (int)__clzll((long long)some) : -1;
    }
    __syncthreads();
    int who = -1;
#pragma unroll
    for (int w = 3; w >= 0; --w) who = hits[w] >= 0 ? hits[w] : who;
    if (who < 0)
#pragma unroll
        for (int w = 0; w < 4; ++w) who = hits[4 + w] >= 0 ? hits[4 + w] : who;
    return who;
}

// Whether a given draft row holds anything above 0; all threads.  A token that was drawn from the row does, so that this is
// met only where the drafted token is none, or was not drawn from it.
template <typename XT>
__device__ bool any_drawn(const DraftVerify &a, int64_t row_q) {
    const XT *d = static_cast<const XT *>(a.draft) + row_q * a.ld_draft;
    bool some = false;
    for (int e = threadIdx.x; e < a.n_vocab; e += 8 * 256) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = act_to_f32(d[e + i * 256 < a.n_vocab ? e + i * 256 : a.n_vocab - 1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) some |= y[i] > 0.f;
    }
    return __syncthreads_or(some) != 0;
}

// The token that follows, and all of a sequence's results: one workgroup, after all tile sums.
template <typename XT, bool PROBS>
__device__ __forceinline__ void pick_token(const DraftVerify &a, const DraftPlan &p, int s, const Pick &pick) {
    const int tid = threadIdx.x, wave = tid >> 6;
    __shared__ double wave_sums[4], before;
    __shared__ int hits[8], found;
    double *tiles = reinterpret_cast<double *>(a.ws + p.off_tiles) + (int64_t)s * p.tiles;
    const float u = a.u[(int64_t)s * (a.max_draft + 1) + a.max_draft];
    const int64_t place = (int64_t)s * (a.max_draft + 1) + tid;
    const int drafted = tid < pick.taken ? a.tokens[(int64_t)s * a.max_draft + tid] : -1;
    int kind = pick.kind, result = pick.token;
    if (PROBS && kind == kMinus && pick.token == kUnseen && !any_drawn<XT>(a, pick.row_q)) kind = kFixed, result = -1;
    // a thread's tiles, next to each other; their sums stay in registers (8 of them: over a million tokens)
    constexpr int kHeld = 8;
    const int each = (p.tiles + 255) / 256, t0 = tid * each, t1 = t0 + each < p.tiles ? t0 + each : p.tiles;
    if (kind != kFixed) {
        double own, run, total, held[kHeld];
        auto sums = [&]() {
            own = 0.0;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) held[i] = i < each && t0 + i < t1 ? sum_of(tiles + t0 + i) : 0.0;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) own += held[i];
            for (int t = t0 + kHeld; t < t1; ++t) own += sum_of(tiles + t);
            run = run_256(own, wave_sums, total);
        };
        sums();
        // Next to nothing is left of p - q (uniform): p itself.  A token that was drawn from q is refused as often as p - q
        // leaves, so this is not met in earnest; what is left then is the rounding of p and q (some 2^-50).
        if (total < 0x1p-32 && kind != kPlain) {
            kind = kPlain;
            for (int t = wave; t < p.tiles; t += 4) {
                const double again = tile_sum<XT, PROBS>(a, pick, kind, t);
                if ((tid & 63) == 0) put_sum(tiles + t, again);
            }
            sums_done();
            sums();
        }
        result = -1;
        if (total > 0.0 && total < __builtin_inf()) {
            const double r = (u > 0.f ? (double)u : 0.0) * total;
            if (tid == thread_at(run, own, r, hits)) {
                double at = run - own, from = at;
                int tile = t0;
                bool passed = false;
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    if (!passed && held[i] > 0.0) tile = t0 + i, from = at, passed = at + held[i] > r;
                    at += held[i];
                }
                for (int t = t0 + kHeld; t < t1 && !passed; ++t) {
                    const double v = sum_of(tiles + t);
                    if (v > 0.0) tile = t, from = at, passed = at + v > r;
                    at += v;
                }
                found = tile, before = from;
            }
            __syncthreads();
            constexpr int kEach = kTile / 256;
            static_assert(kEach == 2, "two tokens a thread");
            const int e = found * kTile + tid * kEach;
            const double base = before;
            Tokens<kEach, XT> t;
            t.load(a, pick, kind, e, 1);
            double w[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) w[i] = t.template left<PROBS>(a, pick, kind, i, e + i);
            own = w[0] + w[1];
            run = base + run_256(own, wave_sums, total);
            if (tid == thread_at(run, own, r, hits)) {
                double at = run - own;
                int hit = 0;
#pragma unroll
                for (int i = kEach - 1; i >= 0; --i) hit = w[i] > 0.0 ? i : hit;      // (the first that holds anything)
                bool passed = false;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    at += w[i];
                    if (!passed && w[i] > 0.0) hit = i, passed = at > r;
                }
                found = e + hit;
            }
            __syncthreads();
            result = found;
        }
    }
    if (tid <= a.max_draft) {
        const int taken = pick.taken;
        a.out[place] = tid < taken ? drafted : tid == taken ? result : -1;
        if (tid == 0) a.n_accepted[s] = taken < 0 ? 0 : taken;
    }
}

// The workgroup of a sequence that is done last takes the token (of logits: draft_stats has set its count to 0; given
// probabilities have no launch before this one that could, and draft_pick follows).
template <typename XT, bool PROBS>
__global__ __launch_bounds__(256, 5) void draft_sums(DraftVerify a, DraftPlan p) {
    const int s = (int)(blockIdx.x / (unsigned)p.sum_parts), g = (int)(blockIdx.x % (unsigned)p.sum_parts);
    __shared__ Pick pick;
    __shared__ bool last;
    decide<XT, PROBS>(a, p, s, pick);
    __syncthreads();
    if (PROBS && g == 0 && threadIdx.x == 0) reinterpret_cast<Pick *>(a.ws + p.off_pick)[s] = pick;
    const Pick mine = uniform(pick);
    if (mine.kind == kFixed) {
        if (!PROBS && g == 0) pick_token<XT, PROBS>(a, p, s, mine);
        return;
    }
    for (int tile = g * 4 + (int)(threadIdx.x >> 6); tile < p.tiles; tile += p.sum_parts * 4) {
        const double sum = tile_sum<XT, PROBS>(a, mine, mine.kind, tile);
        if ((threadIdx.x & 63) == 0) put_sum(reinterpret_cast<double *>(a.ws + p.off_tiles) + (int64_t)s * p.tiles + tile, sum);
    }
    if (PROBS) return;
    sums_done();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(reinterpret_cast<int *>(a.ws + p.off_done) + s * kCountEvery, 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == p.sum_parts - 1;
    sums_done();
    if (!last) return;
    pick_token<XT, PROBS>(a, p, s, mine);
}

template <typename XT>
__global__ __launch_bounds__(256) void draft_pick(DraftVerify a, DraftPlan p) {
    pick_token<XT, true>(a, p, blockIdx.x, uniform(reinterpret_cast<const Pick *>(a.ws + p.off_pick)[blockIdx.x]));
}

DraftPlan draft_plan(int64_t n_seqs, int64_t max_draft, int64_t n_vocab, bool has_draft, int elem_bytes, bool probs) {
    DraftPlan p{};
    const int64_t rows = probs ? 0 : n_seqs * (max_draft + 1 + (has_draft ? max_draft : 0));
    const int64_t ve = 16 / elem_bytes, vecs = (n_vocab + 2 * ve - 2) / ve;      // of the worst alignment
    // one pass a workgroup until there are some 23 workgroups for each of the 256 CUs, then longer chunks (576 rows of 38 passes,
    // us: 4 passes 66.0, 2 67.8, 8 67.6, before the exponentials were as short)
    const int64_t pass = kPass / ve;
    int64_t passes = (vecs + pass - 1) / pass, per = 1;
    while (per < 8 && rows * ((passes + per - 1) / per) > 6000) per *= 2;
    p.chunk_vecs = (int)(per * pass);
    p.chunks = (int)((passes + per - 1) / per);
    p.tiles = (int)((n_vocab + kTile - 1) / kTile);
    p.stat_groups = rows * p.chunks;
    // four tiles a workgroup until they are more than the GPU holds at once (5 for each CU), since each decides anew: 64
    // sequences of 297 tiles in 1280 workgroups 90.3 us, in 640 93.8, in 2560 96.6
    const int64_t whole = (p.tiles + 3) / 4, fill = n_seqs > 0 ? (1280 + n_seqs - 1) / n_seqs : 1;
    p.sum_parts = (int)(whole < fill ? whole : fill);
    p.sum_groups = n_seqs * p.sum_parts;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t from = at;
        at += (bytes + 15) / 16 * 16;
        return from;
    };
    p.off_z = take((size_t)p.stat_groups * 8);
    p.off_max = take((size_t)p.stat_groups * 4);
    p.off_arg = take((size_t)p.stat_groups * 4);
    p.off_tiles = take((size_t)n_seqs * p.tiles * 8);
    p.off_done = take((size_t)n_seqs * kCountEvery * 4);
    p.off_pick = take((size_t)n_seqs * sizeof(Pick));
    p.ws_bytes = at;
    return p;
}

hipError_t launch_draft_verify(const DraftVerify &a, const DraftPlan &p, Act xt, bool probs, hipStream_t s) {
    return with_act(xt, [&](auto tag) -> hipError_t {
        using XT = decltype(tag);
        const unsigned sums = (unsigned)p.sum_groups, seqs = (unsigned)a.n_seqs;
        const hipError_t e = probs ? launch(draft_sums<XT, true>, sums, 256, 0, s, a, p)
                                   : launch(draft_stats<XT>, (unsigned)p.stat_groups, 256, 0, s, a, p);
        if (e != hipSuccess) return e;                           // nothing runs after a launch that failed
        return probs ? launch(draft_pick<XT>, seqs, 256, 0, s, a, p) : launch(draft_sums<XT, false>, sums, 256, 0, s, a, p);
    });
}

}  // namespace q2_0
