// A whole expert layer for few tokens: gate and up products with SiLU, down product, weighted
// sum.
//
//   h[p] = silu(W_gate,e x[t]) * (W_up,e x[t])      for each pair p = (t, u), e = ids[p]
//   y[t] = sum_u weights[t][u] * W_down,e h[p]
//
// Up to kFewPairs pairs it is two launches: moe_up_few and moe_down_few (which also sums).
// Beyond, four: moe_prepare, moe_stream for gate and up, moe_stream for down, moe_sum.
//
// Routing.  In moe_up_few workgroup (rows, p) serves the expert of pair p if p is the first pair that
// chose it, for all pairs that did (or row y of the grid is an expert, where the pairs are the more
// numerous), and finds them with one compare and ballot.  (moe_down_few reads an expert's
// weights once per pair: its workgroup is a token's.)  Beyond few pairs moe_prepare lists every chosen
// expert's pairs once, the experts with the most pairs first, so that no late workgroup has two
// passes and none is empty between: with every workgroup of moe_stream finding its own pairs (2.5 of its
// 17 us) in the experts' order 16 tokens took 54.5 us and 64 took 83.  An expert's weights are loaded once
// a pass, of 4 or 8 of its pairs.  Its passes follow one another in a workgroup, so few experts with many pairs each
// leave most of the chip idle and take what one expert's passes take: 64 tokens with 8 of 8 experts 151 us, with 2 of 8
// 66, where 2 us would read the weights.
//
// Products, exact but for the activations' own rounding and the f32 sums over blocks.  An
// activation is fixed point, 31 bits with its sign, below the largest of its 128 neighbours
// (a block pair): X = x 2^(30-E).  Its four signed base-256 digits, (X + 0x00808080) ^
// 0x00808080 byte by byte, are four A rows of v_mfma_i32_16x16x64_i8; the raw 2-bit codes q,
// 16 weight rows, are B; the accumulator starts at minus the digits' sum over the block, so one
// instruction gives sum (q - 1) digit of a 64-weight block, in integers, for 4 columns x 4
// digits and 16 rows.  Digits join in 32-bit integers and one f32 rounding, times d, and add up in
// f32.  Unpacking 16 codes takes 7 instructions (one AND, three shifts and ANDs), where their
// fp16 form (q - 1 exact in fp16, x as a hi/lo pair) takes 17.  The fixed point costs no accuracy where a sum of
// f32 products would keep it: an element errs by 2^-31 of its largest neighbour, a running f32 sum that holds that neighbour
// by 2^-24 of it a step (against 64 bits the layer errs 1.7e-7, products and sums in f32 1.1e-6).  Only a row whose
// weights skip the neighbour, by many zeros in a row, would keep more of the small ones in f32; the bound is the header's.
//
// Weights.  A wave takes two tiles of 16 rows at a time (gate and up of the same rows, or two
// tiles of down), so that one read of the digits serves both; stages of 8 blocks pass through
// registers (one stage ahead) into its own LDS tile.  Rows may start at any 2-byte address: a
// row's 144 bytes are read as 16-byte pieces from its own start, and where fewer are left
// the last piece ends with the row, so nothing outside the row is touched.
//
// What bounds it, for 128 experts of 768 x 2048 with 8 used, in a graph.  One token 13.9 us (10.6 MB of weights,
// 1.7 us of HBM time): the latency of its dependent steps, ids, weights, products, twice.  Every
// instruction line met first costs a trip to the L2, so loops are kept rolled: unrolled
// (12 KB of code instead of 5) the same launches took 19 us.  16 tokens 44.8 us (110 MB, 18 us): gate and up
// 21 us, of which the stream itself runs at HBM rate between the first stage's arrival (6 us) and
// the first workgroup's end; down 14.5, 1.3 rounds of workgroups of one and a half stages; 7 for
// moe_prepare and moe_sum.  64 tokens 74 us (168 MB, 27 us): VALU issue (~80 % while 16 waves of a CU are
// resident) and 1.5 rounds of workgroups.
#include "layer_common.h"
#include "lds_dma.h"
#include "mat_vec_common.h"

namespace q2_0 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Pairs up to which the two launches for few pairs run.  Experts of 768 x 2048, in us, two launches against four: 8 of
// 128 used by 2 tokens 17.8 / 23.3, 3 tokens 23.2 / 24.5, 4 tokens 24.8 / 25.2, 6 tokens 34.0 / 30.8; 4 of 16 by 6
// tokens 20.6 / 23.3, by 12 32.7 / 28.2; 2 of 8 by 8 tokens 17.4 / 22.2, by 12 26.0 / 27.5.
constexpr int kFewPairs = 24;

constexpr int kMlWaves = 8;
constexpr int kMlSB = 8;                                  // blocks of a stage
constexpr int kMlRow = kMlSB * kBlockBytes;               // LDS bytes per row (36 dwords: 16 rows on distinct banks)
constexpr int kMlTileBytes = kMvTile * kMlRow;
constexpr int kMlChunks = kMlRow / 16;                    // 16-byte pieces per row
constexpr int kMlCH = (kMvTile * kMlChunks + 63) / 64;    // pieces per lane and tile

// Orders a wave's LDS stores and loads that pass data between its lanes (no barrier between).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 16 bytes from a 2-byte aligned address
__device__ __forceinline__ uint4 load_piece(const uint8_t *p) {
    struct __attribute__((packed, aligned(2))) Piece {
        uint32_t v[4];
    };
    const Piece t = *reinterpret_cast<const Piece *>(p);
    return uint4{t.v[0], t.v[1], t.v[2], t.v[3]};
}

// Four consecutive activations from an address aligned to one element, as f32.
template <typename XT>
__device__ __forceinline__ float4_t load_x4(const XT *p) {
    struct __attribute__((packed, aligned(sizeof(XT)))) Four {
        XT v[4];
    };
    const Four t = *reinterpret_cast<const Four *>(p);
    return float4_t{act_to_f32(t.v[0]), act_to_f32(t.v[1]), act_to_f32(t.v[2]), act_to_f32(t.v[3])};
}

// ---- weights: sb (1 .. 8) blocks of MATS tiles through registers into the wave's LDS tiles
template <int MATS>
struct WStage {
    uint4 r[MATS][kMlCH];

    // tile m's rows are rowbytes apart from w[m], which points at the stage's first block
    __device__ __forceinline__ void load(const uint8_t *const (&w)[MATS], int rowbytes, int sb, int lane) {
        const int last = sb * kBlockBytes - 16;           // where a row's last piece starts
#pragma unroll
        for (int t = 0; t < kMlCH; ++t) {
            const int c = t * 64 + lane, pc = 16 * (c % kMlChunks);
            if (c >= kMvTile * kMlChunks || pc >= last + 16) continue;
            const int off = c / kMlChunks * rowbytes + min(pc, last);
#pragma unroll
            for (int m = 0; m < MATS; ++m) r[m][t] = load_piece(w[m] + off);
        }
    }
    __device__ __forceinline__ void park(uint8_t *lds, int sb, int lane) const {
        const int last = sb * kBlockBytes - 16;
#pragma unroll
        for (int t = 0; t < kMlCH; ++t) {
            const int c = t * 64 + lane, pc = 16 * (c % kMlChunks);
            if (c >= kMvTile * kMlChunks || pc >= last + 16) continue;
            uint8_t *d = lds + 16 * c - pc + min(pc, last);
#pragma unroll
            for (int m = 0; m < MATS; ++m, d += kMlTileBytes) {
                if (last % 16 == 0) {
                    *reinterpret_cast<uint4 *>(d) = r[m][t];
                } else {                                  // a row's last pieces overlap; they agree
                    const uint32_t v[4] = {r[m][t].x, r[m][t].y, r[m][t].z, r[m][t].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint16_t *>(d + 2 * i) = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
                }
            }
        }
    }
};

// The four B dwords of a code dword: byte b of dword s is code 4b + s.
__device__ __forceinline__ i32x4_t codes_of(uint32_t cd) {
    constexpr uint32_t m = 0x03030303u;
    return i32x4_t{(int)(cd & m), (int)((cd >> 2) & m), (int)((cd >> 4) & m), (int)((cd >> 6) & m)};
}

// A block pair of one tile (mat_vec_common.h's layout: lp points at the pair in this lane's row): the
// lane's codes and the two scales; the odd block past the row's end (odd false) is not data.
struct WPair {
    i32x4_t b[2];
    float d[2];
    __device__ __forceinline__ WPair(const uint8_t *lp, int g, bool odd) {
        const uint32_t X = *reinterpret_cast<const uint32_t *>(lp + 4 * g);
        const uint32_t Z = *reinterpret_cast<const uint32_t *>(lp + 20 + 4 * g);
        const uint32_t D0 = *reinterpret_cast<const uint32_t *>(lp);
        const uint32_t Y = *reinterpret_cast<const uint32_t *>(lp + 16);
        b[0] = codes_of(__builtin_amdgcn_perm(Y, X, g == 0 ? 0x05040302u : 0x03020100u));
        b[1] = codes_of(Z);
        d[0] = half_bits_to_float(D0 & 0xffffu);
        d[1] = odd ? half_bits_to_float(Y >> 16) : 0.f;
    }
};

// acc + d * (a block's product) from the digits' A operand and the accumulator's start
__device__ __forceinline__ float block_product(i32x4_t x, i32x4_t codes, i32x4_t start, float d, float acc) {
    const i32x4_t v = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, codes, start, 0, 0, 0);
    const float f = __builtin_fmaf((float)((v[0] << 8) + v[1]), 65536.f, (float)((v[2] << 8) + v[3]));
    return __builtin_fmaf(d, f, acc);
}

// ---- activations
// x (finite, |x| < 2^E) as the digits word of round(x 2^sh), sh = 30 - E.
__device__ __forceinline__ uint32_t digits_of(float x, int sh) {
    const int v = (int)__builtin_rintf(__builtin_amdgcn_ldexpf(x, sh));
    return ((uint32_t)v + 0x00808080u) ^ 0x00808080u;
}

// Byte k of each of four words as one word, for k = 0..3.
__device__ __forceinline__ void transpose4(const uint32_t w[4], uint32_t t[4]) {
    const uint32_t lo01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), hi01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t lo23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), hi23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    t[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
    t[1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
    t[2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
    t[3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max_row(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
    return v > o ? v : o;
}

template <int CTRL>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}

// The digits of 16 activations: one lane group's share (index ig) of a block, 8 lanes in a row being
// a block pair, which has one scale.  dig: [digit, highest first][dword]; csum: minus the digits'
// sums over the block; scale: 2^(E-30), NaN where the pair holds inf or NaN.
__device__ __forceinline__ void digitise(const float4_t v[4], i32x4_t dig[4], i32x4_t &csum, float &scale) {
    uint32_t mx = 0;                                      // of |x| as bits: ordered, inf and NaN on top
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float f = v[k / 4][k % 4];                  // (a bit cast of a vector element would read element 0)
        mx = max(mx, __builtin_bit_cast(uint32_t, f) & 0x7fffffffu);
    }
    mx = dpp_max_row<0xb1>(mx);                           // over 8 lanes: quad_perm 1,0,3,2 and 2,3,0,1, half mirror
    mx = dpp_max_row<0x4e>(mx);
    mx = dpp_max_row<0x141>(mx);
    // |x| < 2^E; below 2^-96 the scale stays (f32's subnormals count as nothing)
    const int E = max(-96, mx ? __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, mx)) : -96);
    const bool fin = mx < 0x7f800000u;
    scale = fin ? __builtin_amdgcn_ldexpf(1.f, E - 30) : __builtin_nanf("");
    csum = i32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w[4], t[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) w[b] = digits_of(fin ? v[b][q] : 0.f, 30 - E);
        transpose4(w, t);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            dig[d][q] = (int)t[3 - d];
            csum[d] = __builtin_amdgcn_sdot4((int)t[3 - d], -1, csum[d], false);
        }
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        csum[d] = dpp_add<0xb1>(csum[d]);                 // over the block's four lanes
        csum[d] = dpp_add<0x4e>(csum[d]);
    }
}

// The 16 activations of a row that meet lane group ig's code dword of block blk.
template <typename XT>
__device__ __forceinline__ void load_share(const XT *row, int blk, int ig, float4_t v[4]) {
    const XT *xb = row + blk * kBlockWeights;
    const XT *lo = xb + 8 * half_lo(ig, blk & 1), *hi = xb + 8 * half_hi(ig, blk & 1);
    v[0] = load_x4(lo);
    v[1] = load_x4(lo + 4);
    v[2] = load_x4(hi);
    v[3] = load_x4(hi + 4);
}

// silu(v) = v / (1 + e^-v); the exponent's product with log2 e is carried to f32's last bit.
__device__ __forceinline__ float silu(float v) {
    constexpr float l2e = 1.44269504088896340736f, ln2 = 0.69314718055994530942f;
    const float t = -v * l2e;
    const float lo = __builtin_fabsf(t) < 128.f ? __builtin_fmaf(-v, l2e, -t) : 0.f;   // (beyond: 0, inf or a quotient of 1)
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t) * __builtin_fmaf(lo, ln2, 1.f));
}

// ---- routing of few pairs.  grid.y counts experts (by_expert) or pairs.  The pairs that chose this workgroup's
// expert, in order, into list; returns their number, 0 where there is nothing to do (no such
// expert, nobody chose it, an earlier pair's workgroup serves it).
struct Choice {
    const int32_t *ids;
    int n_expert, n_pairs;
    int by_expert;
    FastDiv used;               // a pair's token: pair / slots per token
};

__device__ __forceinline__ int chosen(const Choice &a, int &e, uint8_t *list, int tid) {
    static_assert(kFewPairs <= 64, "a pair a lane");
    e = a.by_expert ? (int)blockIdx.y : a.ids[blockIdx.y];
    if (e < 0 || e >= a.n_expert) return 0;
    const int lane = tid & 63;
    const bool mine = lane < a.n_pairs && a.ids[min(lane, a.n_pairs - 1)] == e;
    const uint64_t hit = __ballot(mine);
    if (hit == 0 || (!a.by_expert && (int)__ffsll((unsigned long long)hit) - 1 < (int)blockIdx.y)) return 0;
    if (tid < 64 && mine) list[__popcll(hit & (((uint64_t)1 << lane) - 1))] = (uint8_t)lane;
    __syncthreads();
    return (int)__popcll(hit);
}

// ---- gate and up of few pairs.  KS: K slices, one wave each, so that 8/KS waves own a tile of gate
// and up; 4 pairs per pass.  The window's activations are digitised here.
struct MoeUp {
    const uint8_t *w0, *w1;     // gate, up
    int64_t expert_bytes;
    const void *x;
    int64_t ldx;
    Choice c;
    int M, nb;                  // rows and blocks per row
    float *h;                   // [pair][M]
};

template <int KS, typename XT>
__global__ __launch_bounds__(64 * kMlWaves, 4) void moe_up_few(MoeUp a) {
    constexpr int NC = 4;                                 // pairs per pass
    constexpr int XB = 32;                                // blocks of a window of activations
    constexpr int SL = XB / KS;                           // of them, blocks of a wave's slice
    constexpr int SUBS = SL / kMlSB;                      // stages of a slice
    static_assert(XB * 4 * NC == 64 * kMlWaves && SL % kMlSB == 0, "an item a thread, whole stages");

    __shared__ __attribute__((aligned(16))) uint8_t lds_w[kMlWaves][2 * kMlTileBytes];
    __shared__ i32x4_t lds_x[XB * 64];                    // [block][lane] A operands
    __shared__ i32x4_t lds_c[XB * NC];                    // [block][column] minus the digits' sums
    __shared__ float lds_s[XB / 2][NC];                   // scales of a column's block pairs
    __shared__ float lds_red[KS > 1 ? kMlWaves * 2 * 64 : 1];
    __shared__ uint8_t lds_list[kFewPairs];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g = lane >> 4;
    int e;
    const int n = chosen(a.c, e, lds_list, tid);
    if (n == 0) return;

    const int ks = wave % KS;
    const int tile = blockIdx.x * (kMlWaves / KS) + wave / KS;
    const bool mine = tile * kMvTile < a.M;
    const int rowbytes = a.nb * kBlockBytes;
    const int64_t at0 = (int64_t)e * a.expert_bytes + (int64_t)tile * kMvTile * rowbytes;
    const int nwin = (a.nb + XB - 1) / XB;
    const XT *x = static_cast<const XT *>(a.x);
    const int ib = (tid >> 2) % XB, ig = tid & 3, icol = tid / (XB * 4);   // this thread's activations
    const uint8_t *lw = &lds_w[wave][j * kMlRow];

    for (int c0 = 0; c0 < n; c0 += NC) {
        float r[2] = {0.f, 0.f};                          // gate, up: column g of row j
        float4_t xreg[4];
        WStage<2> wreg;
        // step s: stage s % SUBS of window s / SUBS.  A step's loads are issued one step ahead, so
        // step -1 only loads.
#pragma unroll 1
        for (int s = -1, win = 0, sub = -1; s < nwin * SUBS; ++s) {
            const int sb = s < 0 || !mine ? 0 : min(kMlSB, a.nb - (win * XB + ks * SL + sub * kMlSB));
            wave_fence();
            if (sb > 0) wreg.park(lds_w[wave], sb, lane);
            wave_fence();
            if (s >= 0 && sub == 0) {
                if (win) __syncthreads();                 // the window before is read
                i32x4_t dig[4], csum;
                float scale;
                digitise(xreg, dig, csum, scale);
                if ((lane & 7) == 0) lds_s[ib / 2][icol] = scale;
#pragma unroll
                for (int d = 0; d < 4; ++d) lds_x[ib * 64 + ig * 16 + 4 * icol + d] = dig[d];
                if (ig == 0) lds_c[ib * NC + icol] = csum;
                __syncthreads();
            }
            // the next step's loads
            int nsub = sub + 1, nw = win;
            if (nsub == SUBS) nsub = 0, ++nw;
            if (nsub == 0 && nw < nwin) {
#pragma unroll
                for (int k = 0; k < 4; ++k) xreg[k] = float4_t{0.f, 0.f, 0.f, 0.f};
                if (c0 + icol < n && nw * XB + ib < a.nb)
                    load_share(x + a.c.used.div((uint32_t)lds_list[c0 + icol]) * a.ldx, nw * XB + ib, ig, xreg);
            }
            const int nb0 = nw * XB + ks * SL + nsub * kMlSB;
            const int nsb = mine ? min(kMlSB, a.nb - nb0) : 0;
            if (nsb > 0) {
                const uint8_t *const w[2] = {a.w0 + at0 + nb0 * kBlockBytes, a.w1 + at0 + nb0 * kBlockBytes};
                wreg.load(w, rowbytes, nsb, lane);
            }
#pragma unroll 1
            for (int t = 0; 2 * t < sb; ++t) {
                const int blk = ks * SL + sub * kMlSB + 2 * t;
                float acc[2] = {0.f, 0.f};
                const WPair p0(lw + 36 * t, g, 2 * t + 1 < sb), p1(lw + kMlTileBytes + 36 * t, g, 2 * t + 1 < sb);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const i32x4_t av = lds_x[(blk + h) * 64 + lane], cv = lds_c[(blk + h) * NC + g];
                    acc[0] = block_product(av, p0.b[h], cv, p0.d[h], acc[0]);
                    acc[1] = block_product(av, p1.b[h], cv, p1.d[h], acc[1]);
                }
                const float sc = lds_s[blk / 2][g];
                r[0] = __builtin_fmaf(acc[0], sc, r[0]);
                r[1] = __builtin_fmaf(acc[1], sc, r[1]);
            }
            sub = nsub;
            win = nw;
        }
        if (KS > 1) {
            // slice partials -> LDS, added in slice order by slice 0's wave
            lds_red[(wave * 2 + 0) * 64 + lane] = r[0];
            lds_red[(wave * 2 + 1) * 64 + lane] = r[1];
            __syncthreads();
            if (ks == 0) {
#pragma unroll 1
                for (int k = 1; k < KS; ++k) {
                    r[0] += lds_red[((wave + k) * 2 + 0) * 64 + lane];
                    r[1] += lds_red[((wave + k) * 2 + 1) * 64 + lane];
                }
            }
        }
        if (ks == 0 && mine && c0 + g < n)
            a.h[(int64_t)lds_list[c0 + g] * a.M + tile * kMvTile + j] = silu(r[0]) * r[1];
        __syncthreads();      // (the next pass overwrites the window, the scales and lds_red)
    }
}

// ---- down product and weighted sum of few pairs: workgroup (tile, token), a wave per slot of the
// token (slots u, u + 8, .. by wave u), on its own from the hidden activation to the slot's 16
// results; these join in LDS in wave order.
struct MoeDown {
    const uint8_t *w;
    int64_t expert_bytes;
    const float *h;             // [pair][nb * 64]
    const int32_t *ids;
    const float *weights;
    int n_expert, n_used, nb;
    float *y;
    int64_t ldy;
};

__global__ __launch_bounds__(64 * kMlWaves, 4) void moe_down_few(MoeDown a) {
    __shared__ __attribute__((aligned(16))) uint8_t lds_w[kMlWaves][kMlTileBytes];
    __shared__ i32x4_t lds_x[kMlWaves][kMlSB * 16];       // [block][g][digit]
    __shared__ i32x4_t lds_c[kMlWaves][kMlSB];
    __shared__ float lds_s[kMlWaves][kMlSB / 2];
    __shared__ float lds_y[kMlWaves][kMvTile];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g = lane >> 4;
    const int ib = lane >> 2, ig = lane & 3;
    const int rowbytes = a.nb * kBlockBytes, nst = (a.nb + kMlSB - 1) / kMlSB;
    const uint8_t *lw = &lds_w[wave][j * kMlRow];
    float y = 0.f;
#pragma unroll 1
    for (int u = wave; u < a.n_used; u += kMlWaves) {
        const int pair = blockIdx.y * a.n_used + u;
        const int e = __builtin_amdgcn_readfirstlane(a.ids[pair]);
        if (e < 0 || e >= a.n_expert) {
            y = __builtin_nanf("");
            continue;
        }
        const float *hp = a.h + (int64_t)pair * a.nb * kBlockWeights;
        const uint8_t *wt = a.w + (int64_t)e * a.expert_bytes + (int64_t)blockIdx.x * kMvTile * rowbytes;
        float r = 0.f;
        float4_t xreg[4];
        WStage<1> wreg;
#pragma unroll 1
        for (int s = -1; s < nst; ++s) {                  // a stage is loaded a step ahead
            const int sb = s < 0 ? 0 : min(kMlSB, a.nb - s * kMlSB);
            wave_fence();
            if (sb > 0) {
                wreg.park(lds_w[wave], sb, lane);
                i32x4_t dig[4], csum;
                float scale;
                digitise(xreg, dig, csum, scale);
                if (ib < kMlSB) {                         // (lanes 0 .. 31)
#pragma unroll
                    for (int d = 0; d < 4; ++d) lds_x[wave][ib * 16 + ig * 4 + d] = dig[d];
                    if (ig == 0) lds_c[wave][ib] = csum;
                    if ((lane & 7) == 0) lds_s[wave][ib / 2] = scale;
                }
            }
            wave_fence();
            const int n0 = (s + 1) * kMlSB, nsb = min(kMlSB, a.nb - n0);
            if (nsb > 0) {
                const uint8_t *const w[1] = {wt + n0 * kBlockBytes};
                wreg.load(w, rowbytes, nsb, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k) xreg[k] = float4_t{0.f, 0.f, 0.f, 0.f};
                if (ib < nsb) load_share(hp, n0 + ib, ig, xreg);
            }
#pragma unroll 1
            for (int t = 0; 2 * t < sb; ++t) {
                const WPair p(lw + 36 * t, g, 2 * t + 1 < sb);
                float acc = 0.f;
                // (A rows past the four digits repeat them, and every lane group gets the result)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    acc = block_product(lds_x[wave][(2 * t + h) * 16 + 4 * g + (j & 3)], p.b[h], lds_c[wave][2 * t + h], p.d[h], acc);
                r = __builtin_fmaf(acc, lds_s[wave][t], r);
            }
        }
        y = __builtin_fmaf(a.weights[pair], r, y);
    }
    if (g == 0) lds_y[wave][j] = y;
    __syncthreads();
    if (tid < kMvTile) {
        float s = lds_y[0][tid];
#pragma unroll 1
        for (int w = 1; w < min(kMlWaves, a.n_used); ++w) s += lds_y[w][tid];
        a.y[blockIdx.y * a.ldy + blockIdx.x * kMvTile + tid] = s;
    }
}

// ---- more pairs: activations digitised once, in memory.  A row's record of a stage (8 blocks): A
// operands [block][g][digit], 16 bytes each, minus the digits' sums [block] (4 ints), scales
// [block pair].
constexpr int kRecC = kMlSB * 256, kRecS = kRecC + kMlSB * 16, kRec = kRecS + 16;

__host__ __device__ inline int stages(int nb) { return (nb + kMlSB - 1) / kMlSB; }

// Stores one lane group's share (ig) of block blk of a row that has nst records at rec; lane: the
// share's place among the 8 of its block pair.
__device__ __forceinline__ void store_record(uint8_t *rec, int blk, int ig, int lane, const float4_t v[4]) {
    i32x4_t dig[4], csum;
    float scale;
    digitise(v, dig, csum, scale);
    uint8_t *r = rec + (int64_t)(blk / kMlSB) * kRec;
    const int b = blk % kMlSB;
#pragma unroll
    for (int d = 0; d < 4; ++d) *reinterpret_cast<i32x4_t *>(r + b * 256 + ig * 64 + d * 16) = dig[d];
    if (ig == 0) *reinterpret_cast<i32x4_t *>(r + kRecC + b * 16) = csum;
    if (lane == 0) *reinterpret_cast<float *>(r + kRecS + b / 2 * 4) = scale;
}

// What moe_stream is told of its experts: one entry per expert that some pair chose, those with the most
// pairs first, then entries of no pairs; and the pairs, an expert's together.
struct Entry {
    int32_t expert, start, n, unused;
};

struct MoePrepare {
    const void *x;
    int64_t ldx;
    int nb;
    uint8_t *rec;
    const int32_t *ids;
    int n_expert, n_pairs, entries;     // entries: the fewer of experts and pairs
    Entry *entry;
    int32_t *list;
    int entry_blocks, token_blocks;     // workgroups of the entries; of a token's digits
    FastDiv per_token;
};

// Wave r of the first workgroups places the expert r (or the expert of pair r, where pairs are the fewer and r
// is the first that chose it) from the counts of all experts, which every workgroup makes for itself in LDS:
// the sums and ranks do not depend on the order of its atomics.  The others write x's records.
template <typename XT>
__global__ __launch_bounds__(256) void moe_prepare(MoePrepare a) {
    extern __shared__ int cnt[];
    const int tid = threadIdx.x;
    if ((int)blockIdx.x >= a.entry_blocks) {
        const int u = (int)blockIdx.x - a.entry_blocks, token = a.per_token.div((uint32_t)u);
        const int it = (u - token * a.token_blocks) * 256 + tid, blk = it >> 2, ig = it & 3;
        const int nst = stages(a.nb);
        if (blk >= nst * kMlSB) return;
        float4_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = float4_t{0.f, 0.f, 0.f, 0.f};
        if (blk < a.nb) load_share(static_cast<const XT *>(a.x) + token * a.ldx, blk, ig, v);
        store_record(a.rec + (int64_t)token * nst * kRec, blk, ig, it & 7, v);
        return;
    }
    for (int i = tid; i < a.n_expert; i += 256) cnt[i] = 0;
    __syncthreads();
    for (int p = tid; p < a.n_pairs; p += 256) {
        const int e = a.ids[p];
        if (e >= 0 && e < a.n_expert) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    const int lane = tid & 63, r = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(tid >> 6);
    if (r >= a.entries) return;
    const bool by_expert = a.entries == a.n_expert;
    const int e = by_expert ? r : __builtin_amdgcn_readfirstlane(a.ids[r]);
    const int n = e >= 0 && e < a.n_expert ? __builtin_amdgcn_readfirstlane(cnt[e]) : 0;
    int start = 0, rank = 0, active = 0;
    for (int i = lane; i < a.n_expert; i += 64) {
        const int c = cnt[i];
        start += i < e ? c : 0;
        rank += c > n || (c == n && i < e) ? 1 : 0;
        active += c > 0 ? 1 : 0;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        start += __shfl_xor(start, off);
        rank += __shfl_xor(rank, off);
        active += __shfl_xor(active, off);
    }
    if (r >= active && lane == 0) a.entry[r] = Entry{0, 0, 0, 0};
    if (n == 0) return;
    int before = 0;
    for (int b = 0; b < a.n_pairs; b += 64) {
        const bool hit = b + lane < a.n_pairs && a.ids[b + lane] == e;
        const uint64_t m = __ballot(hit);
        if (!by_expert && before == 0 && m && b + (int)__ffsll((unsigned long long)m) - 1 < r) return;   // an earlier pair's
        if (hit) a.list[start + before + (int)__popcll(m & (((uint64_t)1 << lane) - 1))] = b + lane;
        before += (int)__popcll(m);
    }
    if (lane == 0) a.entry[rank] = Entry{e, start, n, 0};
}

struct MoeStream {
    const uint8_t *w0, *w1;     // gate and up, or down (w0)
    int64_t expert_bytes;
    const uint8_t *x;           // records, row r at r * stages(nb) * kRec
    const Entry *entry;
    const int32_t *list;
    FastDiv used;               // a pair's token: pair / slots per token
    int M, nb;
    uint8_t *rec;               // UP: h as records, row = pair
    float *out;                 // otherwise: [pair][M]
};

// CG: groups of 4 pairs per pass.  The activations' operands go from the records straight to LDS
// (two buffers of a stage, loaded a stage ahead), one barrier a stage.  UP turns its 128 rows of
// h, a block pair, into records at once.
template <int CG, bool UP>
__global__ __launch_bounds__(64 * kMlWaves, 4) void moe_stream(MoeStream a) {
    constexpr int NC = 4 * CG;
    static_assert(kMlWaves == kMlSB && kMlWaves * kMvTile == 2 * kBlockWeights, "a wave loads a block; a workgroup's rows are a block pair");

    __shared__ __attribute__((aligned(16))) uint8_t lds_w[kMlWaves][2 * kMlTileBytes];
    __shared__ __attribute__((aligned(16))) i32x4_t lds_x[2][kMlSB * CG * 64];   // [block][column group][lane]
    __shared__ __attribute__((aligned(16))) i32x4_t lds_m[2][64 * CG];           // sums [block][column], scales [column][pair]

    // (through the scalar cache: one entry per workgroup)
    typedef const __attribute__((address_space(4))) Entry *EntryPtr;
    const EntryPtr entry = (EntryPtr)(uintptr_t)(a.entry + blockIdx.y);
    const int e = entry->expert, n = entry->n;
    if (n == 0) return;
    typedef const __attribute__((address_space(4))) int32_t *ListPtr;
    const ListPtr list = (ListPtr)(uintptr_t)(a.list + entry->start);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g = lane >> 4;

    const int unit = blockIdx.x * kMlWaves + wave;        // tile pair of this wave
    const bool mine = unit * (UP ? 1 : 2) * kMvTile < a.M;
    const int rowbytes = a.nb * kBlockBytes;
    const int64_t at0 = (int64_t)e * a.expert_bytes + (int64_t)unit * (UP ? 1 : 2) * kMvTile * rowbytes;
    const uint8_t *const w0 = a.w0 + at0, *const w1 = UP ? a.w1 + at0 : w0 + kMvTile * rowbytes;
    const int nst = stages(a.nb);
    const uint8_t *lw = &lds_w[wave][j * kMlRow];
    const uint32_t lx = (uint32_t)(uintptr_t)&lds_x[0][0], lm = (uint32_t)(uintptr_t)&lds_m[0][0];

    for (int c0 = 0; c0 < n; c0 += NC) {
        const int ncg = min(CG, (n - c0 + 3) / 4);
        // The pass's pairs, through the scalar cache as well: a vector load would have to be waited for together
        // with the weights issued before it, or hold these up.  (Past n they are not this expert's, or not
        // pairs: pick clamps.)
        // (vectors: of an array of integers the compiler made indexed memory)
        static_assert(CG <= 2, "pick");
        const i32x4_t qa = {list[c0], list[c0 + 1], list[c0 + 2], list[c0 + 3]};
        i32x4_t qb = qa;
        if (CG > 1) qb = i32x4_t{list[c0 + 4], list[c0 + 5], list[c0 + 6], list[c0 + 7]};
        const auto pick = [qa, qb, c0, n](int col) {
            const int c = min(col, n - 1 - c0);
            int r = qa[0];
            r = c >= 1 ? qa[1] : r;
            r = c >= 2 ? qa[2] : r;
            r = c >= 3 ? qa[3] : r;
            if (CG > 1) {
                r = c >= 4 ? qb[0] : r;
                r = c >= 5 ? qb[1] : r;
                r = c >= 6 ? qb[2] : r;
                r = c >= 7 ? qb[3] : r;
            }
            return r;
        };
        WStage<2> wreg;
        const auto issue_w = [&](int s) {
            const int sb = mine ? min(kMlSB, a.nb - s * kMlSB) : 0;
            const uint8_t *const w[2] = {w0 + s * kMlRow, w1 + s * kMlRow};
            if (sb > 0) wreg.load(w, rowbytes, sb, lane);
        };
        issue_w(0);           // (first: they need only the expert)
        // where this lane's share of a column's record is (columns past n repeat the last one)
        const auto record = [&](int col) {
            const int q = pick(col);
            return a.x + (int64_t)(UP ? a.used.div((uint32_t)q) : q) * nst * kRec;
        };
        const uint8_t *xs[CG];
#pragma unroll
        for (int c = 0; c < CG; ++c) xs[c] = record(4 * c + j / 4) + wave * 256 + g * 64 + (j & 3) * 16;
        const bool sums = CG == 1 ? lane < 32 : wave == 0;    // wave 0 (CG = 2: and 1) also loads sums and scales
        const uint8_t *ms = sums ? record(lane % NC) + kRecC + lane / NC * 16 : record(lane % NC) + kRecS;
        const auto issue_x = [&](int s, int buf) {
#pragma unroll
            for (int c = 0; c < CG; ++c)
                if (c < ncg) lds_dma16(xs[c] + (int64_t)s * kRec, lx + buf * (uint32_t)sizeof(lds_x[0]) + (wave * CG + c) * 1024);
            if (wave < CG) lds_dma16(ms + (int64_t)s * kRec, lm + buf * (uint32_t)sizeof(lds_m[0]) + wave * 1024);
        };
        float r[2][CG];
#pragma unroll
        for (int c = 0; c < CG; ++c) r[0][c] = r[1][c] = 0.f;
        issue_x(0, 0);
#pragma unroll 1
        for (int s = 0; s < nst; ++s) {
            const int buf = s & 1;
            const int sb = mine ? min(kMlSB, a.nb - s * kMlSB) : 0;
            wave_fence();
            if (sb > 0) wreg.park(lds_w[wave], sb, lane);
            wait_vmcnt<0>();          // this wave's share of the stage's operands (issued before its weights)
            __syncthreads();          // everyone's; and the other buffer is read
            if (s + 1 < nst) {
                issue_x(s + 1, buf ^ 1);
                issue_w(s + 1);
            }
            const i32x4_t *xb = lds_x[buf], *mb = lds_m[buf];
            const float *sc = reinterpret_cast<const float *>(mb + kMlSB * NC);
#pragma unroll 1
            for (int t = 0; 2 * t < sb; ++t) {
                const WPair p0(lw + 36 * t, g, 2 * t + 1 < sb), p1(lw + kMlTileBytes + 36 * t, g, 2 * t + 1 < sb);
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    if (c >= ncg) break;
                    const float scale = sc[4 * (4 * c + g) + t];
                    float acc[2] = {0.f, 0.f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const i32x4_t av = xb[((2 * t + h) * CG + c) * 64 + lane];
                        const i32x4_t cv = mb[(2 * t + h) * NC + 4 * c + g];
                        acc[0] = block_product(av, p0.b[h], cv, p0.d[h], acc[0]);
                        acc[1] = block_product(av, p1.b[h], cv, p1.d[h], acc[1]);
                    }
                    r[0][c] = __builtin_fmaf(acc[0], scale, r[0][c]);
                    r[1][c] = __builtin_fmaf(acc[1], scale, r[1][c]);
                }
            }
        }
        __syncthreads();      // (the stage buffers are read: the next pass, or h, may overwrite them)
        if (UP) {
            float(*hl)[2 * kBlockWeights + 4] = reinterpret_cast<float(*)[2 * kBlockWeights + 4]>(&lds_x[0][0]);
#pragma unroll
            for (int c = 0; c < CG; ++c) hl[4 * c + g][wave * kMvTile + j] = silu(r[0][c]) * r[1][c];   // (0 past M)
            __syncthreads();
            int te = tid;
            asm volatile("" : "+v"(te));      // (its index arithmetic stays here: hoisted out of the passes it spills)
            const int col = te >> 3, b = (te >> 2) & 1, ig = te & 3;
            if (col < min(NC, n - c0)) {
                const float *hb = &hl[col][b * kBlockWeights];
                float4_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = *reinterpret_cast<const float4_t *>(hb + 8 * (k < 2 ? half_lo(ig, b) : half_hi(ig, b)) + 4 * (k & 1));
                store_record(a.rec + (int64_t)pick(col) * stages(a.M / kBlockWeights) * kRec, 2 * blockIdx.x + b, ig,
                             te & 7, v);
            }
            __syncthreads();
        } else if (mine) {
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                const int col = c0 + 4 * c + g;
                if (col >= n) continue;
                float *o = a.out + (int64_t)pick(4 * c + g) * a.M + unit * 2 * kMvTile + j;
                o[0] = r[0][c];
                o[kMvTile] = r[1][c];
            }
        }
    }
}

// y[t] = sum_u weights[t][u] z[(t, u)], in u order; NaN where an id is out of range.  Eight
// slots' loads go out together.
__global__ __launch_bounds__(256) void moe_sum(const float *__restrict__ z, const int32_t *__restrict__ ids,
                                               const float *__restrict__ weights, int n_used, int n_expert, int H,
                                               float *__restrict__ y, int64_t ldy) {
    const int t = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= H) return;
    float s = 0.f;
    for (int u0 = 0; u0 < n_used; u0 += 8) {
        float v[8], w[8];
        int e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int p = t * n_used + min(u0 + k, n_used - 1);
            v[k] = z[(int64_t)p * H + i];
            w[k] = weights[p];
            e[k] = ids[p];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float next = e[k] < 0 || e[k] >= n_expert ? __builtin_nanf("") : __builtin_fmaf(w[k], v[k], s);
            s = u0 + k < n_used ? next : s;
        }
    }
    y[t * ldy + i] = s;
}

static int records(int k) { return stages(k / kBlockWeights) * kRec; }   // bytes of a row's records

size_t moe_layer_ws_bytes(int64_t n_ff, int64_t K, int64_t n_used, int64_t n_tokens) {
    // hidden activations (f32, or records, which are larger), the experts' results, x as records
    const size_t pairs = (size_t)(n_tokens * n_used);
    // (and the experts' entries and pairs, with room for a read of 8 pairs at the last)
    return pairs * ((size_t)records((int)n_ff) + (size_t)K * 4 + sizeof(Entry) + 4) + (size_t)n_tokens * records((int)K) + 32;
}

template <typename XT>
static hipError_t launch_few(const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, const Choice &c, int n_ff, int K,
                             const XT *x, int64_t ldx, const float *weights, int n_used, int n_tokens, float *y, int64_t ldy,
                             void *ws, hipStream_t s) {
    const MoeUp up{wg, wu, (int64_t)n_ff * (K / kBlockWeights) * kBlockBytes, x, ldx, c, n_ff, K / kBlockWeights,
                   static_cast<float *>(ws)};
    const int rows = c.by_expert ? c.n_expert : c.n_pairs, tiles = n_ff / kMvTile;
    // K in slices while that leaves no more workgroups than about one a CU: one token in 4, 2 and 1
    // slices 14.4, 16.4 and 20.5 us, two tokens 18.2, 18.1 and 21.5
    const auto grid = [&](int ks) { return dim3((unsigned)((tiles + kMlWaves / ks - 1) / (kMlWaves / ks)), (unsigned)rows); };
    const auto fits = [&](int ks) { return grid(ks).x * grid(ks).y <= 320; };
    if (fits(4)) moe_up_few<4, XT><<<grid(4), 64 * kMlWaves, 0, s>>>(up);
    else if (fits(2)) moe_up_few<2, XT><<<grid(2), 64 * kMlWaves, 0, s>>>(up);
    else moe_up_few<1, XT><<<grid(1), 64 * kMlWaves, 0, s>>>(up);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const MoeDown down{wd, (int64_t)K * (n_ff / kBlockWeights) * kBlockBytes, up.h, c.ids, weights, c.n_expert, n_used,
                       n_ff / kBlockWeights, y, ldy};
    moe_down_few<<<dim3((unsigned)(K / kMvTile), (unsigned)n_tokens), 64 * kMlWaves, 0, s>>>(down);
    return hipGetLastError();
}

template <int CG>
static void launch_stream(const MoeStream &up, const MoeStream &down, unsigned rows, hipStream_t s) {
    const auto grid = [&](int units) { return dim3((unsigned)((units + kMlWaves - 1) / kMlWaves), rows); };
    moe_stream<CG, true><<<grid(up.M / kMvTile), 64 * kMlWaves, 0, s>>>(up);
    moe_stream<CG, false><<<grid(down.M / kMvTile / 2), 64 * kMlWaves, 0, s>>>(down);
}

hipError_t launch_moe_layer(const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, int n_expert, int n_ff, int K,
                            const void *xv, Act xt, int64_t ldx, const int32_t *ids, const float *weights, int n_used,
                            int n_tokens, float *y, int64_t ldy, void *ws, hipStream_t s) {
    const int n_pairs = n_tokens * n_used;
    // grid rows: one per expert or one per pair, whichever are fewer (those of an expert nobody
    // chose, or of a pair whose expert an earlier one serves, end at once)
    const Choice c{ids, n_expert, n_pairs, n_pairs >= n_expert, FastDiv::make((uint32_t)(n_used > 0 ? n_used : 1))};
    return with_act(xt, [&](auto tag) -> hipError_t {
        using XT = decltype(tag);
        const XT *x = static_cast<const XT *>(xv);
        if (n_pairs > 0 && n_pairs <= kFewPairs)
            return launch_few<XT>(wg, wu, wd, c, n_ff, K, x, ldx, weights, n_used, n_tokens, y, ldy, ws, s);
        uint8_t *const hrec = static_cast<uint8_t *>(ws);
        uint8_t *const xrec = hrec + (int64_t)n_pairs * records(n_ff);
        float *const z = reinterpret_cast<float *>(xrec + (int64_t)n_tokens * records(K));
        if (n_pairs) {
            Entry *const entry = reinterpret_cast<Entry *>(z + (int64_t)n_pairs * K);
            int32_t *const list = reinterpret_cast<int32_t *>(entry + n_pairs);
            const int rows = n_pairs < n_expert ? n_pairs : n_expert, tb = (stages(K / kBlockWeights) * kMlSB * 4 + 255) / 256;
            const MoePrepare prep{x, ldx, K / kBlockWeights, xrec, ids, n_expert, n_pairs, rows, entry, list, (rows + 3) / 4, tb,
                                  FastDiv::make((uint32_t)tb)};
            moe_prepare<XT><<<prep.entry_blocks + n_tokens * tb, 256, (size_t)n_expert * 4, s>>>(prep);
            // (what follows reads experts and pairs from the workspace, so it must not run without them)
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const MoeStream up{wg, wu, (int64_t)n_ff * (K / kBlockWeights) * kBlockBytes, xrec, entry, list, c.used, n_ff,
                               K / kBlockWeights, hrec, nullptr};
            const MoeStream down{wd, nullptr, (int64_t)K * (n_ff / kBlockWeights) * kBlockBytes, hrec, entry, list, c.used, K,
                                 n_ff / kBlockWeights, nullptr, z};
            // 8 pairs a pass where many experts have more than 4.  While all of gate-and-up's workgroups are on the chip at
            // once, two a CU, the call waits for the few experts that take a second pass, so there already at 1.5 pairs an
            // expert on average.  Experts of 768 x 2048, in us with 4 and 8: 8 of 128 used, 16 tokens 44.5 / 45.5, 32 tokens
            // 57.9 / 59.1, 48 tokens 70.2 / 66.3, 64 tokens 80.7 / 72.9; 4 of 60, 16 tokens 28.6 / 29.5, 32 tokens 42.3 /
            // 36.2, 64 tokens 52.7 / 45.6; 4 of 16, 8 tokens 31.6 / 26.5, 64 tokens 90.8 / 71.8.
            const bool at_once = (int64_t)rows * ((n_ff + 127) / 128) <= 512;
            if (2 * n_pairs <= (at_once ? 3 : 5) * n_expert) launch_stream<1>(up, down, (unsigned)rows, s);
            else launch_stream<2>(up, down, (unsigned)rows, s);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        moe_sum<<<dim3((unsigned)((K + 255) / 256), (unsigned)n_tokens), 256, 0, s>>>(z, ids, weights, n_used, n_expert, K, y,
                                                                                     ldy);
        return hipGetLastError();
    });
}

}  // namespace q2_0
