// Expert choice from scores in 64 bits: sigmoid or softmax of the logits, a bias for balance, the best
// groups, the n_used best experts in them and their weights.
//
// One wave per token.  Lane l holds PL consecutive experts (l*PL ..) as unsigned 64-bit keys that
// order as the biased scores do (sign-folded bits of the double, NaN below -inf, 0 for "not to be
// chosen").  Scores are worked out in 64 bits because they decide: two f32 sigmoids of different
// logits, or a score and its bias added in f32, fall on the same or on swapped values some
// once in 10^5 choices, and an expert chosen otherwise is another result.  A round takes the
// wave's largest key as moe_choose does, upper halves first and lower halves only where these are
// equal, and the lowest lane and place among equals is the lowest index.
//
// Groups: where one is the keys of 1, 2, 4 .. lanes, those exchange their two best (8 groups of 32 experts: 3 steps);
// else the keys go through LDS and lane g looks through group g.  A group's rank is the number of groups before it, counted
// with a lane read of each.
//
// What bounds it: a launch and the rounds' dependent steps for few tokens (8 of 128 experts: 5.0 us for one token in a
// graph); instruction issue for many: 4096 tokens of 256 experts take 11.3 us, some 950 instructions a token of which 440 are
// the 8 rounds, where their 4.5 MB would take 0.9.
#include <type_traits>

#include "serve_common.h"

namespace q2_0 {

__device__ __forceinline__ uint64_t order_key64(double v) {
    if (v != v) return 1u;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);    // -0 + 0 = +0
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ double key_value64(uint64_t k) {
    if (k <= 1u) return __builtin_nan("");
    return __builtin_bit_cast(double, (k >> 63) ? (k & 0x7fffffffffffffffull) : ~k);
}

__device__ __forceinline__ uint64_t read_lane64(uint64_t v, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (uint64_t)hi << 32 | lo;
}

// e^x within 5 10^-16 + 1.5 10^-17 |x| of itself (the second is log2 e in 64 bits): 2^n 2^r with n = rint(x log2 e) from the low
// bits of x log2 e + 1.5 2^52, r in [-1/2, 1/2] and the polynomial of degree 10 that meets 2^r at the Chebyshev points.  NaN
// stays NaN; 17 instructions, where the library's function takes 45.
__device__ __forceinline__ double exp64(double x) {
    const double big = 6755399441055744.0, k = 1.4426950408889634074;
    const double v = fmax(fmin(x, 1e4), -1e4);
    const double t = fma(v, k, big), q = t - big;
    const double r = fma(v, k, -q);
    double e = 7.072585985243863e-09;
    e = fma(e, r, 1.0208690571348675e-07);
    e = fma(e, r, 1.3215442586966806e-06);
    e = fma(e, r, 1.5252657258554393e-05);
    e = fma(e, r, 0.00015403530441735424);
    e = fma(e, r, 0.0013333558230168296);
    e = fma(e, r, 0.0096181291076069);
    e = fma(e, r, 0.055504108664447695);
    e = fma(e, r, 0.24022650695910097);
    e = fma(e, r, 0.69314718055995);
    e = fma(e, r, 1.0);
    e = __builtin_amdgcn_ldexp(e, (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
    return x != x ? x : e;
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int off) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, off), hi = (uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), off);
    return (uint64_t)hi << 32 | lo;
}

// the two largest of (b1 >= b2) and (o1 >= o2)
__device__ __forceinline__ void two_largest(uint64_t &b1, uint64_t &b2, uint64_t o1, uint64_t o2) {
    const bool more = o1 > b1;
    const uint64_t low = more ? b1 : o1, next = more ? o2 : b2;  // the lower of the largest, and what the larger one's side has next
    b1 = more ? o1 : b1;
    b2 = low > next ? low : next;
}

__device__ __forceinline__ uint64_t group_key(const ChooseGroups &a, uint64_t b1, uint64_t b2) {
    return order_key64(a.group_top == 2 ? key_value64(b1) + key_value64(b2) : key_value64(b1));
}

template <int PL, typename XT, bool SIGMOID>
__global__ __launch_bounds__(256) void moe_choose_groups(ChooseGroups a) {
    extern __shared__ uint64_t key_lds[];                        // 4 waves x 64 * PL keys, with groups only
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.n_tokens) return;                                 // (no barrier below)
    const XT *row = static_cast<const XT *>(a.logits) + t * a.ld;
    // (a lane past the last expert reads that one: no branches around the loads)
    float v[PL], add[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane * PL + i < a.n_expert ? lane * PL + i : a.n_expert - 1;
        v[i] = act_to_f32(row[e]);
        add[i] = a.bias ? a.bias[e] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = lane * PL + i < a.n_expert ? v[i] : -__builtin_inff();
    // softmax about the largest logit; a row of -inf alone has scores 0
    double m = 0.0, inv = 0.0;
    if (!SIGMOID) {
        float top = v[0];
#pragma unroll
        for (int i = 1; i < PL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
        m = top == -__builtin_inff() ? 0.0 : (double)top;
    }
    double s[PL];
    if (SIGMOID) {
#pragma unroll
        for (int i = 0; i < PL; ++i) s[i] = 1.0 / (1.0 + exp64(-(double)v[i]));
    } else {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            s[i] = exp64((double)v[i] - m);
            sum += s[i];
        }
        sum = wave_sum(sum);
        inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
        for (int i = 0; i < PL; ++i) s[i] *= inv;
    }
    uint64_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane * PL + i;
        const uint64_t k = order_key64(s[i] + (double)add[i]);
        key[i] = e < a.n_expert ? k : 0u;
    }
    if (a.group_lanes > 0) {
        // a group is the keys of a power of two of lanes: its two largest by exchanges, and its value is known to all of them
        uint64_t b1 = key[0], b2 = 0u;
#pragma unroll
        for (int i = 1; i < PL; ++i) two_largest(b1, b2, key[i], 0u);
        for (int off = 1; off < a.group_lanes; off <<= 1) {
            const uint64_t o1 = shfl_xor64(b1, off);
            two_largest(b1, b2, o1, shfl_xor64(b2, off));
        }
        const uint64_t g = group_key(a, b1, b2);
        const int mine = lane / a.group_lanes;
        int rank = 0;
        for (int h = 0; h < a.n_group; ++h) {
            const uint64_t k = read_lane64(g, h * a.group_lanes);
            rank += k > g || (k == g && h < mine);
        }
        if (rank >= a.n_group_used)
#pragma unroll
            for (int i = 0; i < PL; ++i) key[i] = 0u;
    } else if (a.n_group > 1) {
        // groups of any size: through LDS, lane g looks through group g
        uint64_t *mine = key_lds + wave * 64 * PL;
#pragma unroll
        for (int i = 0; i < PL; ++i) mine[lane * PL + i] = key[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        uint64_t g = 0u;
        if (lane < a.n_group) {
            const int n = (int)a.size.d;
            uint64_t b1 = 0u, b2 = 0u;
#pragma unroll 4
            for (int i = 0; i < n; ++i) two_largest(b1, b2, mine[lane * n + i], 0u);
            g = group_key(a, b1, b2);
        }
        int rank = 0;
        for (int h = 0; h < a.n_group; ++h) {
            const uint64_t k = read_lane64(g, h);
            rank += k > g || (k == g && h < lane);
        }
        const uint64_t open = __ballot(lane < a.n_group && rank < a.n_group_used);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = lane * PL + i;
            if (e < a.n_expert && !((open >> a.size.div((uint32_t)e)) & 1)) key[i] = 0u;
        }
    }
    int my_id = 0;         // lane u < n_used: the u-th choice
    for (int u = 0; u < a.n_used; ++u) {
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < PL; ++i) {
            const bool more = key[i] > best;
            best = more ? key[i] : best;
            at = more ? i : at;
        }
        const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
        const uint32_t top = wave_max_u32(hi);
        uint64_t held = __ballot(hi == top);
        if (held & (held - 1)) {                                 // (uniform) equal upper halves: the lower ones decide
            const uint32_t low = wave_max_u32(hi == top ? lo : 0u);
            held = __ballot(hi == top && lo == low);
        }
        const int win = (int)__ffsll((unsigned long long)held) - 1;
        const int id = win * PL + __builtin_amdgcn_readlane(at, win);
        my_id = lane == u ? id : my_id;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (lane == win && i == at) key[i] = 0u;
    }
    // the chosen experts' scores without the bias; one that the bias masks (-inf) weighs nothing
    double w = 0.0;
    if (lane < a.n_used) {
        const double x = (double)act_to_f32(row[my_id]);
        w = SIGMOID ? 1.0 / (1.0 + exp64(-x)) : exp64(x - m) * inv;
        if (a.bias && a.bias[my_id] == -__builtin_inff()) w = 0.0;
    }
    if (a.normalise) {
        double sum = w;                                          // (the lanes from n_used on hold 0)
        for (int off = 1; off < a.n_used; off <<= 1) sum += __shfl_xor(sum, off);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    if (lane < a.n_used) {
        a.ids[t * a.n_used + lane] = my_id;
        a.weights[t * a.n_used + lane] = (float)(w * (double)a.scale);   // rounded to f32 once
    }
}

hipError_t launch_moe_choose_groups(ChooseGroups a, Act xt, bool sigmoid, hipStream_t s) {
    return with_act(xt, [&](auto tag) -> hipError_t {
        using XT = decltype(tag);
        const unsigned groups = (unsigned)((a.n_tokens + 3) / 4);
        auto go = [&](auto pl) {
            constexpr int PL = decltype(pl)::value;
            const int lanes = (int)a.size.d / PL;
            a.group_lanes = a.n_group > 1 && a.size.d % PL == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
            const size_t lds = a.n_group > 1 && !a.group_lanes ? 4 * 64 * PL * sizeof(uint64_t) : 0;
            return launch(sigmoid ? moe_choose_groups<PL, XT, true> : moe_choose_groups<PL, XT, false>, groups, 256, lds, s, a);
        };
        // the smallest register tile that holds a row
        if (a.n_expert <= 64) return go(std::integral_constant<int, 1>{});
        if (a.n_expert <= 128) return go(std::integral_constant<int, 2>{});
        if (a.n_expert <= 256) return go(std::integral_constant<int, 4>{});
        if (a.n_expert <= 512) return go(std::integral_constant<int, 8>{});
        return go(std::integral_constant<int, 16>{});
    });
}

}  // namespace q2_0
