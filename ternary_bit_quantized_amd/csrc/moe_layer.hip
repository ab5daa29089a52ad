// A whole expert layer for few tokens: gate and up products with SiLU, down product, weighted
// sum.
//
//   h[p] = silu(W_gate,e x[t]) * (W_up,e x[t])      for each pair p = (t, u), e = ids[p]
//   y[t] = sum_u weights[t][u] * W_down,e h[p]
//
// Routing needs no table: workgroup (tile, p) serves the expert of pair p if p is the first
// pair that chose it, for all pairs that did; every wave finds them with one compare and
// ballot per 64 ids.  So an expert's weights are read once, whatever number of tokens chose
// it, and a launch covers only experts that were chosen.
//
// Products.  Per 64-weight block d * sum (q - 1) x on the matrix cores (mat_vec_common.h):
// up to NC pairs' activations are the A rows as fp16 hi and lo, 16 weight rows the B columns,
// f32 block sums scaled by d and added in f32.  Activations are scaled to the fp16 range by a
// power of two for each 8 blocks of a pair, so a staging wave needs no other wave's maximum.
//
// Layout.  A wave owns 16 weight rows; stages of 16 blocks pass through registers (one stage
// ahead) into its LDS tile.  Rows may start at any 2-byte address: a row's 18*16 bytes are
// read as 16-byte pieces from its own start; a piece that would pass the slice's end is
// read so that it ends there and shifted down, so nothing outside the row is touched.
//
// What bounds it: the latency of its dependent steps (ids, weights, products; two products)
// for one token, decoding of the weights (~60 instructions per 128 weights x 16 rows) for
// many experts.
#include "layer_common.h"
#include "mat_vec_common.h"

namespace q2_0 {

constexpr int kMlSB = 16;                       // blocks per stage
constexpr int kMlRow = kMlSB * kBlockBytes + 16;  // LDS bytes per row
constexpr int kMlChunks = kMlSB * kBlockBytes / 16;               // 16-byte pieces per row
constexpr int kMlCH = (kMvTile * kMlChunks + 63) / 64;            // pieces per lane
constexpr int kMlMaxPairs = Q2_0_MOE_LAYER_MAX_TOKENS * Q2_0_MOE_LAYER_MAX_USED;

struct MoeLayer {
    const uint8_t *w0, *w1;     // gate and up, or down (w0)
    int64_t expert_bytes;
    const void *x;              // rows of activations
    int64_t ldx;
    const int32_t *ids;
    int n_expert, n_used, n_pairs;
    int M, nb;                  // rows and blocks per row of the matrices
    float *out;                 // [pair][M]
};

struct __attribute__((packed, aligned(2))) Piece {
    uint32_t v[4];
};

// 16 bytes from a 2-byte aligned address
__device__ __forceinline__ uint4 load_piece(const uint8_t *p) {
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

// v shifted down by sh bytes (0 < sh < 16, uniform), zeros coming in
__device__ __forceinline__ uint4 shift_down(uint4 v, int sh) {
    uint32_t d[8] = {v.x, v.y, v.z, v.w, 0u, 0u, 0u, 0u};
    if (sh & 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = d[i + 2], d[i + 2] = 0u;
    if (sh & 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = d[i + 1];
    const uint32_t b = (uint32_t)(8 * (sh & 3));
    uint4 r;
    r.x = __builtin_amdgcn_alignbit(d[1], d[0], b);
    r.y = __builtin_amdgcn_alignbit(d[2], d[1], b);
    r.z = __builtin_amdgcn_alignbit(d[3], d[2], b);
    r.w = __builtin_amdgcn_alignbit(0u, d[3], b);
    return r;
}

// The pairs that chose e, in order, into list (written by wave 0); returns their number, or 0
// where a pair before p chose e too.  Every wave computes the same; a barrier must follow
// before list is read.
__device__ __forceinline__ int pairs_of(const int32_t *__restrict__ ids, int n_pairs, int p, int e, int lane, int wave,
                                        uint16_t *list) {
    int n = 0;
    for (int b = 0; b < n_pairs; b += 64) {
        const int q = b + lane;
        const bool hit = q < n_pairs && ids[q] == e;
        const uint64_t mask = __ballot(hit);
        if (n == 0 && mask != 0 && b + (int)__ffsll((unsigned long long)mask) - 1 < p) return 0;
        if (wave == 0 && hit) list[n + (int)__popcll(mask & (((uint64_t)1 << lane) - 1))] = (uint16_t)q;
        n += (int)__popcll(mask);
    }
    return n;
}

// NC: pairs per pass.  UP: waves 0, 1 take rows of gate, waves 2, 3 the same rows of up, and
// out is silu(gate) * up; otherwise the four waves take four tiles of w0.
template <int NC, bool UP, typename XT>
__global__ __launch_bounds__(256) void moe_products(MoeLayer a) {
    constexpr int NR = 2 * NC;
    constexpr int XI = kMlSB * 8 * NC / 256 > 0 ? kMlSB * 8 * NC / 256 : 1;   // activation items per thread
    constexpr int TILES = UP ? 2 : 4;

    __shared__ __attribute__((aligned(16))) uint8_t lds_w[4][kMvTile * kMlRow];
    __shared__ __attribute__((aligned(16))) half8_t lds_x[kMlSB * 8 * NR];
    __shared__ int lds_e[2][NC];                    // exponents of the stage's two 8-block halves
    __shared__ float lds_gate[UP ? 2 * NC * kMvTile : 1];
    __shared__ uint16_t lds_list[kMlMaxPairs];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g = lane >> 4;
    const int p = blockIdx.y;
    const int e = a.ids[p];
    if (e < 0 || e >= a.n_expert) return;
    const int n = pairs_of(a.ids, a.n_pairs, p, e, lane, wave, lds_list);
    if (n == 0) return;
    __syncthreads();

    const int tile = blockIdx.x * TILES + (UP ? (wave & 1) : wave);
    const uint8_t *w = (UP && wave >= 2 ? a.w1 : a.w0) + (int64_t)e * a.expert_bytes +
                       (int64_t)tile * kMvTile * a.nb * kBlockBytes;
    const int rowbytes = a.nb * kBlockBytes;
    const int nstage = (a.nb + kMlSB - 1) / kMlSB;
    const XT *x = static_cast<const XT *>(a.x);

    uint4 wreg[kMlCH];
    XItem xreg[XI];
    // activation item of this thread: (column, block, mfma, group) with 128 items a column, so
    // a wave's 64 items are 8 whole blocks of one column
    const int it = tid & 127;
    const int ib = it >> 3, imu = (it >> 2) & 1, ig = it & 3;
    const PairMasks pm;
    const uint32_t sel = (g == 0) ? 0x05040302u : 0x03020100u;
    const uint8_t *lw_row = &lds_w[wave][j * kMlRow];

    for (int c0 = 0; c0 < n; c0 += NC) {
        const int nc = min(NC, n - c0);
        const auto issue = [&](int st) {
            const int sb = min(kMlSB, a.nb - st * kMlSB);
            const int bytes = sb * kBlockBytes;
#pragma unroll
            for (int t = 0; t < kMlCH; ++t) {
                const int c = t * 64 + lane;
                const int r = c / kMlChunks, at = 16 * (c % kMlChunks);
                uint4 v = {0u, 0u, 0u, 0u};
                if (r < kMvTile && at < bytes)
                    v = load_piece(w + r * rowbytes + st * (kMlSB * kBlockBytes) + min(at, bytes - 16));
                wreg[t] = v;
            }
#pragma unroll
            for (int i = 0; i < XI; ++i) {
                const int col = (tid >> 7) + 2 * i;
                xreg[i] = XItem{};
                if (col < nc && ib < sb) {
                    const int q = lds_list[c0 + col];
                    const XT *xb = x + (int64_t)(UP ? q / a.n_used : q) * a.ldx + (st * kMlSB + ib) * kBlockWeights + 4 * imu;
                    xreg[i] = XItem{load_x4(xb + 8 * half_lo(ig, ib & 1)), load_x4(xb + 8 * half_hi(ig, ib & 1))};
                }
            }
        };
        const auto park = [&](int st) {
            const int bytes = min(kMlSB, a.nb - st * kMlSB) * kBlockBytes;
            const int sh = (16 - bytes % 16) % 16;      // of the piece that passes the end
#pragma unroll
            for (int t = 0; t < kMlCH; ++t) {
                const int c = t * 64 + lane;
                const int r = c / kMlChunks, at = 16 * (c % kMlChunks);
                uint4 v = wreg[t];
                if (sh) {
                    const uint4 d = shift_down(v, sh);
                    const bool cut = at < bytes && at + 16 > bytes;
                    v.x = cut ? d.x : v.x;
                    v.y = cut ? d.y : v.y;
                    v.z = cut ? d.z : v.z;
                    v.w = cut ? d.w : v.w;
                }
                if (r < kMvTile) *reinterpret_cast<uint4 *>(&lds_w[wave][r * kMlRow + at]) = v;
            }
#pragma unroll
            for (int i = 0; i < XI; ++i) {
                const int col = (tid >> 7) + 2 * i;
                if (col >= NC) break;
                float mx = fmaxf(max_abs4(xreg[i].a), max_abs4(xreg[i].c));
#pragma unroll
                for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
                const int ex = column_exponent(mx);
                if (lane == 0) lds_e[(tid >> 6) & 1][col] = ex;
                store_x_item(xreg[i], ex, lds_x + ((ib * 2 + imu) * 4 + ig) * NR + 2 * col);
            }
        };

        float r0 = 0.f, r1 = 0.f;       // columns 2g and 2g + 1 of row j
        issue(0);
        for (int st = 0; st < nstage; ++st) {
            park(st);
            __syncthreads();
            if (st + 1 < nstage) issue(st + 1);
            const int sb = min(kMlSB, a.nb - st * kMlSB);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int np = min(4, (sb - 8 * hf + 1) / 2);      // block pairs of this half
                float acc0[2] = {0.f, 0.f}, acc1[2] = {0.f, 0.f};
                for (int q = 0; q < np; ++q)
                    mv_block_pair<NC>(lw_row + 36 * (4 * hf + q), lds_x + (8 * (8 * hf + 2 * q) + g) * NR + (j % NR), g,
                                      sel, pm, acc0, acc1);
                r0 += __builtin_amdgcn_ldexpf(acc0[0] + acc1[0], -lds_e[hf][min(2 * g, NC - 1)]);
                if (NC > 1) r1 += __builtin_amdgcn_ldexpf(acc0[1] + acc1[1], -lds_e[hf][min(2 * g + 1, NC - 1)]);
            }
            __syncthreads();
        }
        const int row = tile * kMvTile + j;
        if (UP) {
            float *gate = lds_gate + (wave & 1) * NC * kMvTile + j;
            if (wave < 2) {
                if (2 * g < NC) gate[2 * g * kMvTile] = r0;
                if (2 * g + 1 < NC) gate[(2 * g + 1) * kMvTile] = r1;
            }
            __syncthreads();
            if (wave >= 2) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = 2 * g + i;
                    if (col >= nc) continue;
                    const float gt = gate[col * kMvTile], up = i ? r1 : r0;
                    a.out[(int64_t)lds_list[c0 + col] * a.M + row] = gt / (1.f + expf(-gt)) * up;
                }
            }
        } else {
            if (2 * g < nc) a.out[(int64_t)lds_list[c0 + 2 * g] * a.M + row] = r0;
            if (2 * g + 1 < nc) a.out[(int64_t)lds_list[c0 + 2 * g + 1] * a.M + row] = r1;
        }
        // (the next pass's first barrier separates these reads of lds_gate from its writes)
    }
}

// y[t] = sum_u weights[t][u] z[(t, u)], in u order; NaN where an id is out of range.
__global__ __launch_bounds__(256) void moe_sum(const float *__restrict__ z, const int32_t *__restrict__ ids,
                                               const float *__restrict__ weights, int n_used, int n_expert, int H,
                                               float *__restrict__ y, int64_t ldy) {
    const int t = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= H) return;
    float s = 0.f;
    for (int u = 0; u < n_used; ++u) {
        const int p = t * n_used + u, e = ids[p];
        s = e < 0 || e >= n_expert ? __builtin_nanf("") : __builtin_fmaf(weights[p], z[(int64_t)p * H + i], s);
    }
    y[t * ldy + i] = s;
}

size_t moe_layer_ws_bytes(int64_t n_ff, int64_t K, int64_t n_used, int64_t n_tokens) {
    return (size_t)(n_tokens * n_used) * (size_t)(n_ff + K) * 4;
}

template <typename XT>
static void launch_products(bool up, int nc, const MoeLayer &a, hipStream_t s) {
    const dim3 grid((unsigned)(a.M / (kMvTile * (up ? 2 : 4))), (unsigned)a.n_pairs);
    if (up) {
        if (nc <= 1) moe_products<1, true, XT><<<grid, 256, 0, s>>>(a);
        else if (nc <= 2) moe_products<2, true, XT><<<grid, 256, 0, s>>>(a);
        else if (nc <= 4) moe_products<4, true, XT><<<grid, 256, 0, s>>>(a);
        else moe_products<8, true, XT><<<grid, 256, 0, s>>>(a);
    } else {
        if (nc <= 1) moe_products<1, false, XT><<<grid, 256, 0, s>>>(a);
        else if (nc <= 2) moe_products<2, false, XT><<<grid, 256, 0, s>>>(a);
        else if (nc <= 4) moe_products<4, false, XT><<<grid, 256, 0, s>>>(a);
        else moe_products<8, false, XT><<<grid, 256, 0, s>>>(a);
    }
}

hipError_t launch_moe_layer(const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, int n_expert, int n_ff, int K,
                            const void *x, Act xt, int64_t ldx, const int32_t *ids, const float *weights, int n_used,
                            int n_tokens, float *y, int64_t ldy, void *ws, hipStream_t s) {
    const int n_pairs = n_tokens * n_used;
    float *h = static_cast<float *>(ws);
    float *z = h + (int64_t)n_pairs * n_ff;
    if (n_pairs) {
        const MoeLayer up{wg, wu, (int64_t)n_ff * (K / kBlockWeights) * kBlockBytes, x, ldx, ids, n_expert, n_used,
                          n_pairs, n_ff, K / kBlockWeights, h};
        // (an expert meets at most n_tokens pairs unless a token names it twice)
        hipError_t e = with_act(xt, [&](auto tag) -> hipError_t {
            launch_products<decltype(tag)>(true, n_tokens, up, s);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
        const MoeLayer down{wd, nullptr, (int64_t)K * (n_ff / kBlockWeights) * kBlockBytes, h, n_ff, ids, n_expert,
                            n_used, n_pairs, K, n_ff / kBlockWeights, z};
        launch_products<float>(false, n_tokens, down, s);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    moe_sum<<<dim3((unsigned)((K + 255) / 256), (unsigned)n_tokens), 256, 0, s>>>(z, ids, weights, n_used, n_expert, K, y,
                                                                                   ldy);
    return hipGetLastError();
}

}  // namespace q2_0
