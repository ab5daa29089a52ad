// Expert choice: the n_used largest router logits of a token and their softmax weights.
//
// One wave per token.  Lane l holds PL consecutive logits (experts l*PL ..), as unsigned
// keys that order as the logits do: sign-folded f32 bits (-0 as +0), NaN below -inf, 0 for
// "no expert" and for one already taken.  A round takes the wave's largest key; among lanes
// that hold it the lowest lane, and in that lane the lowest place, is the lowest index.  The
// wave maximum is six DPP steps (~150 cycles a round with the ballot), where lane
// exchanges through LDS would take some 700.
//
// What bounds it: a launch for few tokens (8 of 128 experts: 2.9 us for one token in a graph); for many its
// rounds: 4096 tokens take 4.2 us, their 2.4 MB would take 0.5.
#include <type_traits>

#include "layer_common.h"

namespace q2_0 {

__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 1u;
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);   // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);           // -inf: 0x007fffff
}

template <int PL, typename XT>
__global__ __launch_bounds__(256) void moe_choose(const XT *__restrict__ logits, int64_t ld, int64_t n_tokens,
                                                  int n_expert, int n_used, int normalise, int32_t *__restrict__ ids,
                                                  float *__restrict__ weights) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= n_tokens) return;
    const XT *row = logits + t * ld;
    float v[PL];
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane * PL + i;
        v[i] = e < n_expert ? act_to_f32(row[e]) : -__builtin_inff();
        key[i] = e < n_expert ? order_key(v[i]) : 0u;
    }
    int my_id = 0;         // lane u < n_used: the u-th choice
    float my_v = -__builtin_inff();
    for (int u = 0; u < n_used; ++u) {
        uint32_t best = key[0];
        int at = 0;
        float bv = v[0];
#pragma unroll
        for (int i = 1; i < PL; ++i) {
            const bool more = key[i] > best;
            best = more ? key[i] : best;
            at = more ? i : at;
            bv = more ? v[i] : bv;
        }
        const uint32_t top = wave_max_u32(best);
        const int win = (int)__ffsll((unsigned long long)__ballot(best == top)) - 1;
        const int id = win * PL + __builtin_amdgcn_readlane(at, win);
        const float val = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, bv), win));
        if (lane == u) {
            my_id = id;
            my_v = val;
        }
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (lane == win && i == at) key[i] = 0u;
    }
    // softmax in f32 about the largest logit; -inf everywhere leaves nothing: weights 0
    const float m = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_v), 0));
    const bool none = m == -__builtin_inff();
    const float e = none ? 0.f : expf(my_v - m);
    float sum = lane < n_used ? e : 0.f;
    if (!normalise && !none) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (lane * PL + i < n_expert) sum += expf(v[i] - m);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane < n_used) {
        ids[t * n_used + lane] = my_id;
        weights[t * n_used + lane] = none ? 0.f : e / sum;
    }
}

hipError_t launch_moe_choose(const void *logits, Act xt, int64_t ld, int64_t n_tokens, int n_expert, int n_used,
                             int normalise, int32_t *ids, float *weights, hipStream_t s) {
    return with_act(xt, [&](auto tag) -> hipError_t {
        using XT = decltype(tag);
        const XT *x = static_cast<const XT *>(logits);
        const dim3 grid((unsigned)((n_tokens + 3) / 4));
        auto go = [&](auto pl) {
            moe_choose<decltype(pl)::value, XT><<<grid, 256, 0, s>>>(x, ld, n_tokens, n_expert, n_used, normalise, ids,
                                                                     weights);
        };
        // the smallest register tile that holds a row
        if (n_expert <= 64) go(std::integral_constant<int, 1>{});
        else if (n_expert <= 128) go(std::integral_constant<int, 2>{});
        else if (n_expert <= 256) go(std::integral_constant<int, 4>{});
        else if (n_expert <= 1024) go(std::integral_constant<int, 16>{});
        else go(std::integral_constant<int, 128>{});
        return hipGetLastError();
    });
}

}  // namespace q2_0
