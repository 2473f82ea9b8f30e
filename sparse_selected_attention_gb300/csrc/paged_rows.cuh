// Attention of one token per row over a paged sequence, row by row.
//
//   s_c = scale * q . K_c,  O = sum_c 2^(s_c log2e - m) V_c / sum_c 2^(s_c log2e - m)
//
// One pass over the cache with a running maximum m and sum.  It is bound by
// reading the cache: 2 D + 16 bytes per (cell, KV head) against 4 D flops per
// query head, 23 flops per byte at 12 heads.
//
// Work.  A row's cells are taken in units (32 cells of 128 dims or 16 of 256:
// 8 KB of codes).  The units of all rows are cut into equal shares, one per CTA
// of each KV head, so one long row or a ragged batch fills the chip alike and
// the share does not depend on the table's width.  The KV heads of a share are
// neighbouring CTAs: they walk the same cells together, so that a cell's
// scales, eight bytes per head, come from DRAM once for all heads of a 32-byte
// sector.  A share that holds all of a row writes its output; a row that spans
// CTAs leaves one partial per CTA in the workspace (values, maximum, sum), and
// a second launch joins them.  Each CTA finds its place by summing the rows'
// lengths itself, which costs one pass over seq_lens and saves a launch.
// (Shares by warp instead of by CTA, without block barriers: 202 us for 61 rows
// of up to 32 K cells where this took 187, the partials being four times as
// many.)  Consecutive rows of one sequence go to paged_group.cu where that saves
// enough (take_groups).
//
// 61 rows of up to 32 K cells, 48/4 heads of 128, 1.1 GB: 205 us, 5.4 TB/s; the
// same launch without the arithmetic 176 us.  A row of 321 cells alone: 8 us, all
// of it latency (10.5 us in a table of 32 K cells, with the join's launch).
//
// A unit.  The query heads of one KV head are the M side (padded to 16) of
// m16n8k16 products, cells are N of Q.K and the contraction of P.V.  (tcgen05
// would want the codes as fp16 in shared memory, a round trip of four bytes
// per code; here they go from shared memory to fragments.)  The warps of a CTA
// take a row's units in turn.  Each streams its units through a ring of two
// stages, filled by TMA boxes of 32 or 16 rows x 128 bytes and eight-byte
// cp.async for the scales; the next unit's copies are in flight while one is
// computed, across rows too.  The boxes carry the 128-byte swizzle, and cells
// and dims are assigned to lanes so that no fragment read meets a bank twice:
//   lane (g, r) = (lane / 4, lane % 4) holds cells 4 r .. 4 r + 3 of each 16:
//   column n of score tile j is cell 16 (j / 2) + 2 n + j % 2;
//   K (eight bytes a read): dims 32 b + 8 r + 4 h + {0, 2 | 1, 3} of k-step (b, h);
//   V (transposed 16 x 16 byte matrices): tile t holds dims 8 t .. 8 t + 7.
// Codes become fp16 integers by or-ing 0x6400 to the code + 128 (1024 + 128 +
// code).  For K the 1152 may stay: the accumulators then start at -1152 * sum q,
// so the products give q . code per scale group, and the group's scale
// multiplies in fp32 (compute_unit says when).  For V it is subtracted, and the
// scales go to the weights, a set of fp16 weights per scale group (weight x
// scale in fp32, rounded once: a first rounding of the weight alone would add as
// much again, for 2 us of 196).  So that the products use fp16's range whatever
// the scales are, the running maximum is one of weight x scale, up to a power of
// two per cell: m is the largest s_c log2e + e_c, e_c the exponent of cell c's
// largest V scale.  (One exponent per unit where its cells' are alike, and this where
// not: 204 us for the rows below, where this takes 205 by one path.)
#pragma once

#include <cuda.h>

#include <algorithm>
#include <cfloat>

#include "paged_attn.cuh"

namespace qsa {
namespace {

constexpr int NW = 4;           // warps per CTA, where a row's are not one
constexpr int CTAS_PER_SM = 2;  // 255 registers a thread
constexpr int MAX_CTAS = 152 * CTAS_PER_SM;
static_assert(MAX_CTAS <= MAX_PARTS && WHOLE == 4 * NW, "shared with the join and the groups");
// A warp per row, six to an SM, where the table holds up to SMALL cells and there
// are more rows and KV heads than CTAs of four warps; of more than two units,
// twice as many.  Four warps and one, us: 156 rows, 48/8 heads of 128, one cell 23,
// 17, 64 cells 26, 21, 128 cells 27, 30; 24/4 heads of 256, one cell 17, 11, 64 cells
// 19, 17, but 80 rows of 64 cells 13, 15.
constexpr int SMALL = 64, SMALL_PER_SM = 6;
constexpr int TILE = 4096;      // a unit's K or V codes
// Fewest units of a share, one per warp: finer ones would only add partials.
constexpr int MIN_SHARE = NW;

// S = head_dim / 128.
template <int S>
struct Shape {
    static constexpr int D = 128 * S, UNIT = 32 / S;  // cells of a unit
    static constexpr int NJ = 4 / S, NK = 2 / S;      // score tiles of eight cells, halves of 16
    static constexpr unsigned FULL = S == 1 ? 0xffffffffu : 0xffffu;
};

// Bytes 0 and 2 (or 1 and 3) of w, as fp16 1152 + code.
__device__ __forceinline__ uint32_t even_codes(uint32_t w) { return tc::prmt(w ^ 0x80808080u, 0x64646464u, 0x4240); }
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return tc::prmt(w ^ 0x80808080u, 0x64646464u, 0x4341); }

// Two 16 x 16 byte matrices of V, cells as rows, from lanes 0-15's and lanes
// 16-31's row addresses: registers 0 and 2 hold cells 4 r .. 4 r + 3 of dim g
// of the first and the second, registers 1 and 3 those of dim g + 8.
__device__ __forceinline__ void load_v(uint32_t (&w)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int head, int cell, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(head), "r"(cell), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool pred) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(pred ? 8 : 0));
}

// Shared memory of a CTA of W warps.
template <int S, int W>
struct Smem {
    uint8_t tile[W][2][2][TILE];                  // stage, K or V: [S][UNIT][128] codes; 1024-byte aligned
    uint2 scale[W][2][2][Shape<S>::UNIT];         // four fp16 per cell
    uint4 q[8 * S][32];                            // Q fragments by k-step and lane
    float bias[4][8][4];                           // -1152 * sum of q over a scale group, as accumulators: heads g, g, g + 8, g + 8
    float qinv[16];                                // 2^-e of a head's scaled query
    alignas(16) float ve[W][Shape<S>::UNIT], vw[W][Shape<S>::UNIT];  // of the unit at hand, by cell: e_c and 2^-e_c
    float o[W][16][128];                          // 128 dims of the warps' values, at the end of a segment
    float m[W][16], l[W][16], f[W][16];
    uint64_t bar[W][2];
    long long together[W], padded[W], scan[W];
    long long total, before;                       // units of all rows; of the rows before `row`
    int row, left;                                 // the share's units
};

// Sums the rows' units and finds the row that holds unit share * range, of
// `ranges` shares.
// Each thread takes a run of rows.  share 0: no row has more than WHOLE units,
// and each is taken whole (64 rows of 40 cells in a wide table, 48/4 heads of 256:
// 12 us; 23 us where a share took four of them, one after the other).  False: the
// rows are taken by groups (block 0: there are none).
template <int S, class A>
__device__ __forceinline__ bool find_start(const A &a, Smem<S, NW> &sh, int kvh, int range, int ranges, int block, int &share) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = (a.n_tokens + NW * 32 - 1) / (NW * 32);
    const int t0 = min(tid * run, a.n_tokens), t1 = min(t0 + run, a.n_tokens);
    bool bad = false;
    long long mine = 0, padded = 0, together = 0;
    int most = 0;
    auto pad = [](int u) { return (u + MIN_SHARE - 1) & -MIN_SHARE; };
    for (int t = t0; t < t1; ++t) {
        int row;
        const int u = units_of<S>(row_len(a, t, kvh, row, bad));
        mine += u;
        padded += pad(u);
        most = max(most, u);
        if (block && group_start(a.rows, t, block) == t) {
            int longest = u;
            const int end = group_end(a, t, block), same = __ldg(a.rows + t);
            for (int i = t + 1; i < end && __ldg(a.rows + i) == same; ++i) longest = max(longest, units_of<S>(row_len(a, i, kvh, row, bad)));
            together += longest;
        }
    }
    if (bad && blockIdx.x == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
    long long s = mine, sp = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o), up = __shfl_up_sync(0xffffffffu, sp, o);
        if (lane >= o) {
            s += u;
            sp += up;
        }
    }
    if (block) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) together += __shfl_xor_sync(0xffffffffu, together, o);
    }
    if (lane == 31) {
        sh.scan[warp] = s;
        sh.padded[warp] = sp;
        sh.together[warp] = together;
    }
    share = 0;
    if (!__syncthreads_or(most > WHOLE)) return true;
    long long total = 0, before = 0, groups = 0, total_padded = 0, before_padded = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) {
            before += sh.scan[w];
            before_padded += sh.padded[w];
        }
        total += sh.scan[w];
        total_padded += sh.padded[w];
        groups += sh.together[w];
    }
    if (block && take_groups<S>(a, total, groups, true)) return false;
    before += s - mine;
    before_padded += sp - padded;
    const long long per = (total + ranges - 1) / ranges;
    share = (int)max(per, (long long)MIN_SHARE);
    // Where CTAs are to spare, no share goes over a row's end: the rows' units
    // count as padded to whole shares (four rows of 321 cells, 24/2 heads of 256:
    // 13.0 us, 17.0 us without).
    const bool aligned = share == MIN_SHARE && total_padded <= (long long)share * ranges;
    if (aligned) {
        total = total_padded;
        before = before_padded;
        mine = padded;
    }
    const long long x0 = (long long)share * range;
    if (x0 >= before && x0 < before + mine) {
        for (int t = t0;; ++t) {
            int row;
            const int u = units_of<S>(row_len(a, t, kvh, row, bad)), v = aligned ? pad(u) : u;
            if (x0 < before + v) {
                sh.row = t;
                sh.before = before;
                sh.left = aligned ? (int)min((long long)share, before + u - x0) : (int)min((long long)share, total - x0);
                break;
            }
            before += v;
        }
    }
    if (tid == 0) sh.total = total;
    __syncthreads();
    return true;
}

// The query heads of (row t, KV head kvh) as A fragments in shared memory,
// fp16, with the sums that undo the codes' 1152.  bf16 queries are scaled by
// a power of two per head where they would leave the fp16 range; fp16 ones
// are used as they are.  A negative softmax scale flips their sign.  A warp
// takes every W-th head; the loads are apart from the rest, so that a
// segment's can be in flight while the one before ends.
template <int S, int W>
struct Query {
    static constexpr int D = Shape<S>::D, N = D / 32, H = 16 / W;
    uint32_t raw[H][N / 2];

    __device__ __forceinline__ void load(const qsa_paged_attn_args &a, int t, int kvh, int per) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int h = warp + i * W;
            const size_t at = ((size_t)t * a.n_q_heads + (size_t)kvh * per + h) * D + lane * N;
#pragma unroll
            for (int e = 0; e < N / 2; ++e) raw[i][e] = 0u;
            if (h < per && QSA_IN(at + N - 1, (size_t)a.n_tokens * a.n_q_heads * D)) {
                const uint16_t *src = static_cast<const uint16_t *>(a.q) + at;
                if constexpr (N == 4)
                    *reinterpret_cast<uint2 *>(raw[i]) = __ldg(reinterpret_cast<const uint2 *>(src));
                else
                    *reinterpret_cast<uint4 *>(raw[i]) = __ldg(reinterpret_cast<const uint4 *>(src));
            }
        }
    }

    __device__ __forceinline__ void store(const qsa_paged_attn_args &a, Smem<S, W> &sh) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int h = warp + i * W;
            float x[N], top = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint16_t v = (uint16_t)(raw[i][e / 2] >> (16 * (e & 1)));
                x[e] = a.dtype == QSA_F16 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
                top = fmaxf(top, fabsf(x[e]));
            }
            int ex = 0;
            if (a.dtype != QSA_F16) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                ex = head_sum_exponent(top);
            }
            const float f = (a.softmax_scale < 0.0f ? -1.0f : 1.0f) * exp2i(ex);
            if (lane == 0) sh.qinv[h] = exp2i(-ex);
            __half v[N];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[e] = __float2half_rn(x[e] * f);
                sum += __half2float(v[e]);
            }
            // A scale group is D/4 dims, eight lanes.
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if ((lane & 7) == 0)
                *reinterpret_cast<float2 *>(&sh.bias[lane >> 3][h & 7][2 * (h >> 3)]) = make_float2(-1152.0f * sum, -1152.0f * sum);
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                const int d = lane * N + e, ks = 2 * (d >> 5) + ((d >> 2) & 1), r = (d >> 3) & 3;
                uint32_t *dst = reinterpret_cast<uint32_t *>(&sh.q[ks][(h & 7) * 4 + r]) + (h >> 3);
                dst[0] = h2u(__halves2half2(v[e], v[e + 2]));
                dst[2] = h2u(__halves2half2(v[e + 1], v[e + 3]));
            }
        }
    }
};

template <int S>
struct State {
    float o[16 * S][4];  // o[t][0..1]: head g, dims 8 t + 2 r, 8 t + 2 r + 1; o[t][2..3]: head g + 8
    float m[2], l[2];
    uint32_t k;  // the largest |K scale| that this lane has seen, as bits, in two halves
};

// Folds one staged unit into the state.  vmask: the unit's valid cells.  EXACT:
// scores are summed over K's codes, not over 1152 + codes from -1152 sum q with
// sixteen times the rounding, and the products weight x scale go in in two parts
// of 11 bits, not in one.  Long rows average both (off by 2e-7 of lse, and by
// 1.2 times the output's own rounding), and would pay 2.6 to 7% for exact codes
// alone (61 rows of 48/4 heads of 128; 90 rows of 18 K cells, one head of 256).
// Of short ones, a few cells carry the result (1.2e-6 of lse, 1.5 times the
// output's rounding), and the time is latency: so EXACT goes with short tables
// (short rows of a wide table go with the long ones), and of listed rows and drafts
// with rows of up to WHOLE units (61 listed rows of up to 2 K cells 48 us, 47 without).
template <int S, bool EXACT>
__device__ __forceinline__ void compute_unit(const uint8_t *K, uint32_t V, const uint2 *KS, const uint2 *VS, const uint4 (*q)[32],
                                             const float (*bias)[8][4], float *ve, float *vw, unsigned vmask, State<S> &st,
                                             const float (&sl2)[2]) {
    constexpr int NJ = Shape<S>::NJ, NK = Shape<S>::NK, UNIT = Shape<S>::UNIT;
    const int lane = threadIdx.x & 31, g = lane >> 2, r = lane & 3;
    // Row 2 g of K with the swizzle of its first 16 bytes for this lane, and row 2 g + 1.
    const uint32_t kt = tc::smem_u32(K) + 2 * g * 128 + ((r & 1) << 3);
    const uint32_t keven = kt + (((r >> 1) ^ ((2 * g) & 7)) << 4), kodd = kt + 128 + (((r >> 1) ^ ((2 * g + 1) & 7)) << 4);

    const __half2 off = u2h(0x64806480u);  // 1152
    auto even = [&](uint32_t w) { return h2u(__hsub2(u2h(even_codes(w)), off)); };
    auto odd = [&](uint32_t w) { return h2u(__hsub2(u2h(odd_codes(w)), off)); };
    auto k_even = [&](uint32_t w) { return EXACT ? even(w) : even_codes(w); };
    auto k_odd = [&](uint32_t w) { return EXACT ? odd(w) : odd_codes(w); };

    // A cell that is not there has scales of 0.
    const uint2 kown = KS[lane % UNIT];
    st.k = __vimax3_u16x2(st.k, kown.x & 0x7FFF7FFFu, kown.y & 0x7FFF7FFFu);
    const int own = scale_exponent(VS[lane % UNIT]);
    ve[lane % UNIT] = (float)own;
    vw[lane % UNIT] = exp2i(-own);
    __syncwarp();

    // Scores: per scale group S 32-dim blocks of two k-steps from -1152 sum q,
    // then the scale.
    float2 s[NJ][2];
#pragma unroll
    for (int j = 0; j < NJ; ++j) s[j][0] = s[j][1] = make_float2(0.0f, 0.0f);
    uint4 ks[NK][2];  // scales of cells 16 kk + 4 r .. + 3
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i) ks[kk][i] = *reinterpret_cast<const uint4 *>(KS + 16 * kk + 4 * r + 2 * i);
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
        const float4 c0 = EXACT ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *reinterpret_cast<const float4 *>(bias[gr][g]);
        float acc[NJ][4];
#pragma unroll
        for (int bb = 0; bb < S; ++bb) {
            const int b = gr * S + bb, half = b >> 2, bh = b & 3;  // of all dims; of the 128 of a tile half
            const uint4 q0 = q[2 * b][lane], q1 = q[2 * b + 1][lane];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                uint32_t w0, w1;
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                             : "=r"(w0), "=r"(w1)
                             : "r"((((j & 1) ? kodd : keven) ^ (bh << 5)) + (j >> 1) * 16 * 128 + half * UNIT * 128)
                             : "memory");
                if (bb == 0)
                    mma16816(acc[j], q0, k_even(w0), k_odd(w0), c0.x, c0.y, c0.z, c0.w);
                else
                    mma16816(acc[j], q0, k_even(w0), k_odd(w0), acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
                mma16816(acc[j], q1, k_even(w1), k_odd(w1), acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
            }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            // Cells 4 r + j % 2 and two on: the first or second half of each 16 bytes.
            const uint4 &lo = ks[j >> 1][0], &hi = ks[j >> 1][1];
            const uint32_t w0 = (j & 1) ? (gr >> 1 ? lo.w : lo.z) : (gr >> 1 ? lo.y : lo.x);
            const uint32_t w1 = (j & 1) ? (gr >> 1 ? hi.w : hi.z) : (gr >> 1 ? hi.y : hi.x);
            const float2 f = (gr & 1) ? make_float2(__high2float(u2h(w0)), __high2float(u2h(w1)))
                                      : make_float2(__low2float(u2h(w0)), __low2float(u2h(w1)));
            s[j][0] = __ffma2_rn(make_float2(acc[j][0], acc[j][1]), f, s[j][0]);
            s[j][1] = __ffma2_rn(make_float2(acc[j][2], acc[j][3]), f, s[j][1]);
        }
    }
    if (vmask != Shape<S>::FULL) {
        const unsigned mine = vmask >> (4 * r);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = 16 * (j >> 1) + (j & 1);
            if (!((mine >> c) & 1u)) s[j][0].x = s[j][1].x = -CUDART_INF_F;
            if (!((mine >> (c + 2)) & 1u)) s[j][0].y = s[j][1].y = -CUDART_INF_F;
        }
    }

    // In base 2, with the V exponents.  The reference maximum moves only when a
    // unit exceeds it by 2^SLACK, so the values are rarely rescaled.  Weights
    // 2^(s_c log2e - m), in fp32: weight times V scale is rounded to fp16, once (by
    // at most 2^-11 of itself).  EXACT rounds a weight's argument at its own size,
    // the others at that of score plus exponent (2^-21 of a weight where that is 8
    // to 16).
    const float2 f[2] = {make_float2(sl2[0], sl2[0]), make_float2(sl2[1], sl2[1])};
    float2 w[NJ][2], sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    float mx[2] = {-CUDART_INF_F, -CUDART_INF_F}, al[2];
    auto of_cells = [&](const float *x, int j) {  // of cells 4 r + j % 2 and two on
        const float4 b = *reinterpret_cast<const float4 *>(x + 16 * (j >> 1) + 4 * r);
        return (j & 1) ? make_float2(b.y, b.w) : make_float2(b.x, b.z);
    };
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 t = __ffma2_rn(s[j][e], f[e], of_cells(ve, j));
            mx[e] = max3(mx[e], t.x, t.y);
            if constexpr (!EXACT) s[j][e] = t;
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float mn = mx[e] > st.m[e] + SLACK ? mx[e] : st.m[e];
        al[e] = ex2(st.m[e] - mn);
        st.m[e] = mn;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float2 less = make_float2(-st.m[e], -st.m[e]);
            float2 p;
            if constexpr (EXACT)
                p = __ffma2_rn(s[j][e], f[e], __fadd2_rn(of_cells(ve, j), less));
            else
                p = __fadd2_rn(s[j][e], less);
            w[j][e] = __fmul2_rn(make_float2(ex2(p.x), ex2(p.y)), of_cells(vw, j));
            sum[e] = __fadd2_rn(sum[e], w[j][e]);
        }
#pragma unroll
    for (int e = 0; e < 2; ++e) st.l[e] = fmaf(st.l[e], al[e], sum[e].x + sum[e].y);
    if (__any_sync(0xffffffffu, al[0] != 1.0f || al[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < 16 * S; ++i) {
            st.o[i][0] *= al[0];
            st.o[i][1] *= al[0];
            st.o[i][2] *= al[1];
            st.o[i][3] *= al[1];
        }
    }

    // This lane's row address of V's matrices: 128 dims, cells 0-31 by lane; or
    // cells 0-15 by lane % 16, lanes 16-31 sixteen dims on.
    const uint32_t vrow = S == 1 ? V + lane * 128 + ((lane & 7) << 4) : V + (lane & 15) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
    uint4 vs[NK][2];
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i) vs[kk][i] = *reinterpret_cast<const uint4 *>(VS + 16 * kk + 4 * r + 2 * i);
    auto pv = [&](float (&o)[4], const uint4 &p, const uint4 &rest, uint32_t w) {
        mma16816(o, p, even(w), odd(w), o[0], o[1], o[2], o[3]);
        if constexpr (EXACT) mma16816(o, rest, even(w), odd(w), o[0], o[1], o[2], o[3]);
    };
#pragma unroll
    for (int gr = 0; gr < 4; ++gr) {
        uint4 p[NK], rest[NK];
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            const uint4 &lo = vs[kk][0], &hi = vs[kk][1];
            const uint32_t l0 = gr >> 1 ? lo.y : lo.x, l1 = gr >> 1 ? lo.w : lo.z;  // cells 4 r and on
            const uint32_t h0 = gr >> 1 ? hi.y : hi.x, h1 = gr >> 1 ? hi.w : hi.z;
            auto scale = [&](uint32_t x) { return (gr & 1) ? __high2float(u2h(x)) : __low2float(u2h(x)); };
            const float2 f02 = make_float2(scale(l0), scale(h0)), f13 = make_float2(scale(l1), scale(h1));
            auto scaled = [&](float2 x, float2 f, uint32_t &high, uint32_t &low) {
                const float2 y = __fmul2_rn(x, f);
                const __half2 h = __floats2half2_rn(y.x, y.y);
                high = h2u(h);
                if constexpr (EXACT) low = h2u(__floats2half2_rn(y.x - __low2float(h), y.y - __high2float(h)));
            };
            scaled(w[2 * kk][0], f02, p[kk].x, rest[kk].x);
            scaled(w[2 * kk][1], f02, p[kk].y, rest[kk].y);
            scaled(w[2 * kk + 1][0], f13, p[kk].z, rest[kk].z);
            scaled(w[2 * kk + 1][1], f13, p[kk].w, rest[kk].w);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t v[4];
            if constexpr (S == 1) {  // 16 dims of both halves of the cells
                const int c = 2 * gr + i;
                load_v(v, vrow ^ (c << 4));
                pv(st.o[2 * c], p[0], rest[0], v[0]);
                pv(st.o[2 * c + 1], p[0], rest[0], v[1]);
                pv(st.o[2 * c], p[NK - 1], rest[NK - 1], v[2]);
                pv(st.o[2 * c + 1], p[NK - 1], rest[NK - 1], v[3]);
            } else {  // 32 dims
                const int c = 2 * (gr & 1) + i, t = 16 * (gr >> 1) + 4 * c;
                load_v(v, (vrow ^ (c << 5)) + (gr >> 1) * UNIT * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k) pv(st.o[t + k], p[0], rest[0], v[k]);
            }
        }
    }
}

// The units of a warp in order, across rows: unit u of row t is the next
// one whose copies start.  The row after, and the page of the next unit, are
// loaded a step before they are needed.
struct Feed {
    int t, trow, len, sure, u, end;  // units up to `end` of row t are this CTA's
    int left;                        // its units in the rows after
    int next_trow, next_len, next_sure;
    int slot;                        // this lane's page of the sequence for unit u
    int page;                        // and its table entry
    int ahead, ahead_t, ahead_u;     // of a list: the entry for the unit after, if it is unit ahead_u of row ahead_t
};

// WHOLE_ROWS: no row is shared out.
template <int S, int W, bool WHOLE_ROWS, class A>
__global__ void __launch_bounds__(W * 32, W == 1 ? SMALL_PER_SM : CTAS_PER_SM)
    paged_attn_kernel(const A a, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, int block) {
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem<S, W> &sh = *reinterpret_cast<Smem<S, W> *>(raw);
    constexpr int D = Shape<S>::D, UNIT = Shape<S>::UNIT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, r = lane & 3;
    const int per = a.n_q_heads / a.n_kv_heads, page_shift = 31 - __clz(a.page_size);
    if (lane == 0) {
        tc::mbar_init(tc::smem_u32(&sh.bar[warp][0]), 1);
        tc::mbar_init(tc::smem_u32(&sh.bar[warp][1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_previous_grid();
    allow_dependent_launch();
    const int kvh = blockIdx.x % a.n_kv_heads, range = blockIdx.x / a.n_kv_heads, ranges = gridDim.x / a.n_kv_heads;
    const Work work(a.workspace, MAX_CTAS, per);
    // This CTA's units: `left` of them from unit u0 of row t on, or of whole
    // rows every ranges-th from row `range`.
    int share = 0, t = range, u0 = 0, left = 0x7fffffff;
    bool none = false;
    if constexpr ((LISTED<A> || TREE<A>) && !WHOLE_ROWS) none = a.taken && __ldcg(a.taken + kvh);
    if constexpr (!WHOLE_ROWS) none = none || !find_start<S>(a, sh, kvh, range, ranges, block, share);
    const int step = share ? 1 : ranges;
    if (share) {
        const long long x = (long long)share * range, total = sh.total;
        none = x >= total;
        if (!none) {
            left = sh.left;
            t = sh.row;
            u0 = (int)(x - sh.before);
        }
    } else {
        none |= t >= a.n_tokens;
    }
    if (none) {
        if (tid == 0 && !WHOLE_ROWS) work.part[blockIdx.x] = Part{-1, 0, 0, 0};
        return;
    }
    bool bad = false, dead = false;
    uint32_t phase = 0;   // parity of each stage's next completion, one bit per stage
    uint32_t flying = 0;  // stages with copies in flight
    Feed f;
    f.t = t;
    f.len = row_len(a, t, kvh, f.trow, f.sure, bad);
    int nu = units_of<S>(f.len);
    f.end = min(nu, u0 + left);
    f.left = left - (f.end - u0);
    f.u = u0 + warp;
    f.next_len = f.next_trow = f.next_sure = 0;
    f.ahead_t = -1;
    auto peek = [&] {
        if (f.left > 0 && f.t + step < a.n_tokens) f.next_len = row_len(a, f.t + step, kvh, f.next_trow, f.next_sure, bad);
    };
    // Moves on to the next row that has a unit for this warp.
    auto settle = [&] {
        while (f.u >= f.end && f.left > 0 && f.t + step < a.n_tokens) {
            f.t += step;
            f.len = f.next_len;
            f.trow = f.next_trow;
            f.sure = f.next_sure;
            f.end = min(units_of<S>(f.len), f.left);
            f.left -= f.end;
            f.u = warp;
            peek();
        }
        int j = (f.u * UNIT + lane % UNIT) >> page_shift;
        if constexpr (LISTED<A>) {
            // The list's entry and then the table's are two loads one after the other;
            // the first of them is made a unit before.
            auto entry = [&](int t, int u) {
                const int i = (u * UNIT + lane % UNIT) >> page_shift;
                return i < a.width ? __ldg(a.lists + ((size_t)t * a.n_kv_heads + kvh) * a.width + i) : -1;
            };
            const bool known = f.ahead_t == f.t && f.ahead_u == f.u;
            j = f.u >= f.end || f.u * UNIT + lane % UNIT >= f.len ? -1 : known ? f.ahead : entry(f.t, f.u);
            bad |= j < -1 || j >= a.max_pages;
            f.slot = j < a.max_pages ? j : -1;
            const bool same = f.u + W < f.end;
            f.ahead_t = same ? f.t : f.t + step;
            f.ahead_u = same ? f.u + W : warp;
            if (same || (f.left > 0 && f.ahead_t < a.n_tokens)) f.ahead = entry(f.ahead_t, f.ahead_u);
        }
        f.page = f.u < f.end && j >= 0 && j < a.max_pages ? __ldg(a.page_table + (size_t)f.trow * a.max_pages + j) : -1;
    };
    // Starts the copies of unit f.u into a stage and moves on; returns the
    // unit's valid cells (none past the last unit).
    auto issue = [&](int stage) -> unsigned {
        const int c = f.u * UNIT + lane % UNIT;
        bool in = f.u < f.end && c < f.len;
        if constexpr (LISTED<A>) in = in && f.slot >= 0 && (f.slot << page_shift) + (c & (a.page_size - 1)) < f.sure;
        const bool held = in && f.page >= 0 && f.page < a.n_pages;  // alike for a page's cells up to the last that is `in`
        if constexpr (TREE<A>) in = in && (c < f.sure || (tree_bits(a, f.t, c, f.sure) & 1u));
        const bool ok = in && held;
        bad |= in && !held;
        const unsigned vmask = __ballot_sync(0xffffffffu, ok) & Shape<S>::FULL;
        const size_t cell = held ? ((size_t)f.page << page_shift) + (c & (a.page_size - 1)) : 0;
        const size_t si = (cell * a.n_kv_heads + kvh) * 4;
        const bool sok = ok && QSA_IN(si + 3, (size_t)a.n_pages * a.page_size * a.n_kv_heads * 4);
        if constexpr (S == 1) {
            cp_async8(tc::smem_u32(&sh.scale[warp][stage][0][lane]), a.ksc + (sok ? si : 0), sok);
            cp_async8(tc::smem_u32(&sh.scale[warp][stage][1][lane]), a.vsc + (sok ? si : 0), sok);
        } else {  // lanes 0-15 K's, lanes 16-31 V's
            cp_async8(tc::smem_u32(&sh.scale[warp][stage][lane >> 4][lane & 15]), (lane & 16 ? a.vsc : a.ksc) + (sok ? si : 0), sok);
        }
        asm volatile("cp.async.commit_group;\n" ::);
        // A box starts on the first cell of a page or of a unit in one.
        const int cell16 = __shfl_sync(0xffffffffu, (int)cell, 16);
        if (vmask && !dead) {
            flying |= 1u << stage;
            if (lane == 0) {
                const uint32_t bar = tc::smem_u32(&sh.bar[warp][stage]);
                const uint32_t k = tc::smem_u32(sh.tile[warp][stage][0]), v = k + TILE;
                if constexpr (S == 2) {
                    expect_tx(bar, 2 * TILE);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        tma_box(k + half * TILE / 2, &kmap, 128 * half, kvh, (int)cell, bar);
                        tma_box(v + half * TILE / 2, &vmap, 128 * half, kvh, (int)cell, bar);
                    }
                } else if (a.page_size >= UNIT) {
                    expect_tx(bar, 2 * TILE);
                    tma_box(k, &kmap, 0, kvh, (int)cell, bar);
                    tma_box(v, &vmap, 0, kvh, (int)cell, bar);
                } else {  // two pages of 16 cells
                    const bool lo = vmask & 0xFFFFu, hi = vmask >> 16;
                    expect_tx(bar, (lo && hi ? 2 : 1) * TILE);
                    if (lo) {
                        tma_box(k, &kmap, 0, kvh, (int)cell, bar);
                        tma_box(v, &vmap, 0, kvh, (int)cell, bar);
                    }
                    if (hi) {
                        tma_box(k + TILE / 2, &kmap, 0, kvh, cell16, bar);
                        tma_box(v + TILE / 2, &vmap, 0, kvh, cell16, bar);
                    }
                }
            }
        }
        f.u += W;
        settle();
        return vmask;
    };

    Query<S, W> q;
    q.load(a, t, kvh, per);
    peek();
    settle();
    q.store(a, sh);
    int stage = 0;
    unsigned vmask = 0;
    bool ahead = false;  // the next unit's copies have been started
    Part part{-1, 0, 0, 0};
    __syncthreads();  // the query fragments

    for (bool first = true;; first = false) {
        // Segment: units u0 .. u1-1 of row t; this warp's are u0 + warp, + W ...
        const int u1 = min(nu, u0 + left), n_units = u1 - u0;
        const int n = n_units > warp ? (n_units - warp + W - 1) / W : 0;
        // |scale| in base 2, floored at the smallest normal float: with scale
        // 0 the weights are uniform and a masked -inf stays -inf.
        const float sl2[2] = {fmaxf(fabsf(a.softmax_scale) * LOG2E * sh.qinv[g], 1.17549435e-38f),
                              fmaxf(fabsf(a.softmax_scale) * LOG2E * sh.qinv[g + 8], 1.17549435e-38f)};
        State<S> st;
#pragma unroll
        for (int i = 0; i < 16 * S; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.0f;
        st.m[0] = st.m[1] = -CUDART_INF_F;
        st.l[0] = st.l[1] = 0.0f;
        st.k = 0u;
        for (int i = 0; i < n; ++i) {
            if (!ahead) vmask = issue(stage);
            const unsigned vnext = issue(stage ^ 1);
            ahead = true;
            asm volatile("cp.async.wait_group 1;\n" ::);
            if (vmask) {
                if (!dead && !tc::mbar_wait_bounded(tc::smem_u32(&sh.bar[warp][stage]), (phase >> stage) & 1u, tc::WAIT_LIMIT)) {
                    dead = true;
                    if (lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_TIMEOUT);
                }
                dead = __any_sync(0xffffffffu, dead);
                if (!dead) {
                    phase ^= 1u << stage;
                    flying &= ~(1u << stage);
                }
                __syncwarp();
                const uint8_t *k = sh.tile[warp][stage][0];
                auto compute = [&](auto exact) {
                    compute_unit<S, decltype(exact)::value>(k, tc::smem_u32(k) + TILE, sh.scale[warp][stage][0], sh.scale[warp][stage][1], sh.q,
                                                            sh.bias, sh.ve[warp], sh.vw[warp], vmask, st, sl2);
                };
                if constexpr ((LISTED<A> || TREE<A>) && !WHOLE_ROWS) {
                    if (nu <= WHOLE)
                        compute(std::true_type{});
                    else
                        compute(std::false_type{});
                } else {
                    compute(std::integral_constant<bool, WHOLE_ROWS>{});
                }
            }
            __syncwarp();  // every lane has read the stage before it is filled again
            vmask = vnext;
            stage ^= 1;
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], o);
            st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], o);
        }
        // A cell with an infinite or NaN K scale scores NaN, and its row's heads
        // are NaN: said here, once, since the scale times the codes' sum can be
        // -inf, a cell left out.
        if (__any_sync(0xffffffffu, max(st.k & 0xFFFFu, st.k >> 16) >= 0x7C00u)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                st.m[e] = fmaxf(st.m[e], -FLT_MAX);
                st.l[e] = CUDART_NAN_F;
            }
        }
        left -= n_units;
        const int next = t + step;
        const bool more = left > 0 && next < a.n_tokens;
        if (more) q.load(a, next, kvh, per);
        __syncthreads();  // all warps are done with the query, and with the values of the segment before
        if (r == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sh.m[warp][g + 8 * e] = st.m[e];
                sh.l[warp][g + 8 * e] = st.l[e];
            }
        }
        if (more) q.store(a, sh);
        const bool whole = n_units == nu;
        const size_t at = (size_t)blockIdx.x * 2 + (first && u0 > 0 ? 0 : 1);
        // Join the warps' states, 128 dims at a time.
#pragma unroll
        for (int half = 0; half < S; ++half) {
            // Value (h, d) of a warp sits at d ^ 8 (h % 4) of its row: the lanes
            // of an 8-byte store then meet each bank once, and reads of
            // consecutive d stay consecutive.
            if (half) __syncthreads();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = (8 * i + 2 * r) ^ (8 * (g & 3));
                *reinterpret_cast<float2 *>(&sh.o[warp][g][d]) = make_float2(st.o[16 * half + i][0], st.o[16 * half + i][1]);
                *reinterpret_cast<float2 *>(&sh.o[warp][g + 8][d]) = make_float2(st.o[16 * half + i][2], st.o[16 * half + i][3]);
            }
            __syncthreads();
            if (half == 0) {
                if (tid < 16) {
                    float M = -CUDART_INF_F, L = 0.0f, w[W];
#pragma unroll
                    for (int p = 0; p < W; ++p) M = fmaxf(M, sh.m[p][tid]);
#pragma unroll
                    for (int p = 0; p < W; ++p) {
                        w[p] = sh.m[p][tid] == -CUDART_INF_F ? 0.0f : exp2f(sh.m[p][tid] - M);
                        L += w[p] * sh.l[p][tid];
                    }
                    const float inv = whole ? (M == -CUDART_INF_F ? 0.0f : 1.0f / L) : 1.0f;
#pragma unroll
                    for (int p = 0; p < W; ++p) sh.f[p][tid] = w[p] * inv;
                    if (tid < per) {
                        if (!whole)
                            *reinterpret_cast<float2 *>(work.ml + (at * per + tid) * 2) = make_float2(M, L);
                        else if (a.lse)
                            a.lse[(size_t)t * a.n_q_heads + kvh * per + tid] = lse_of(M, L);
                    }
                }
                __syncthreads();
            }
            // A warp takes 64 dims of every ROWS-th head, BATCH heads at a time
            // with their gates on the way together.
            constexpr int BATCH = 4, COLS = W > 1 ? 2 : 1, ROWS = W / COLS;
            const size_t row0 = (size_t)t * a.n_q_heads + (size_t)kvh * per;
            for (int dc = warp % COLS; dc < 2; dc += COLS) {
                const int d = 64 * dc + 2 * lane, dd = 128 * half + d;
                for (int h0 = warp / COLS; h0 < per; h0 += ROWS * BATCH) {
                    float2 gate[BATCH], y[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int h = h0 + ROWS * k;
                        gate[k] = a.gate && whole && h < per && QSA_IN((row0 + h) * D + dd + 1, (size_t)a.n_tokens * a.n_q_heads * D)
                                      ? __ldg(reinterpret_cast<const float2 *>(a.gate + (row0 + h) * D + dd))
                                      : make_float2(0.0f, 0.0f);
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int h = min(h0 + ROWS * k, per - 1), pd = d ^ (8 * (h & 3));
                        y[k] = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int p = 0; p < W; ++p) {
                            const float w = sh.f[p][h];
                            y[k] = __ffma2_rn(*reinterpret_cast<const float2 *>(&sh.o[p][h][pd]), make_float2(w, w), y[k]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int h = h0 + ROWS * k;
                        if (h >= per) break;
                        if (!whole) {
                            *reinterpret_cast<float2 *>(work.o + (at * per + h) * D + dd) = y[k];
                        } else if (QSA_IN((row0 + h) * D + dd + 1, (size_t)a.n_tokens * a.n_q_heads * D)) {
                            if (a.gate) y[k] = make_float2(gated(y[k].x, gate[k].x), gated(y[k].y, gate[k].y));
                            store_out(a, (row0 + h) * D + dd, y[k]);
                        }
                    }
                }
            }
        }
        if (!whole && u0 == 0) part = Part{t, 1 + (nu - u1 + share - 1) / share, 1, 0};
        if (!more) break;
        t = next;
        u0 = 0;
        int trow;
        nu = units_of<S>(row_len(a, t, kvh, trow, bad));
    }
    asm volatile("cp.async.wait_group 0;\n" ::);
    if (flying) {  // after a time-out: copies in flight land before this CTA's shared memory is given up
        for (int i = 0; i < 2; ++i)
            if ((flying >> i) & 1u) tc::mbar_wait_bounded(tc::smem_u32(&sh.bar[warp][i]), (phase >> i) & 1u, tc::DRAIN_LIMIT);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
    if (tid == 0 && !WHOLE_ROWS) work.part[blockIdx.x] = part;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Codes [cells, heads, D] in boxes of `cells` cells x one head x 128 dims.
inline cudaError_t encode_boxes(CUtensorMap &map, const qsa_paged_attn_args &a, const int8_t *codes, int cells) {
    const EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_kv_heads, (cuuint64_t)a.n_pages * a.page_size};
    const cuuint64_t strides[2] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_kv_heads * a.head_dim};
    const cuuint32_t box[3] = {128, 1, (cuuint32_t)cells}, ones[3] = {1, 1, 1};
    const CUresult e = fn(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t *>(codes), dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Boxes of a unit's cells, or a page's, if fewer.
template <int S>
cudaError_t encode(CUtensorMap &map, const qsa_paged_attn_args &a, const int8_t *codes) {
    return encode_boxes(map, a, codes, std::min(a.page_size, Shape<S>::UNIT));
}

// Joins the partials of a row that spans CTAs, where there are no groups: part p of the
// one that starts in CTA x is slot 1 of that CTA, then slot 0 of the next ones of its
// KV head.  A block takes its heads, as many as fit; few rows have many parts, which G
// sets of threads share, and a block for each head.  (Of 244 rows of 2 K cells, cold,
// blocks that go round over a list of the CTAs in which rows start took 12 us, this 7.)
constexpr int JOIN_THREADS = 1024;
template <int S, int G>
constexpr int JOIN_HEADS = JOIN_THREADS / (64 * S * G);  // of a block, at most
template <int S, int G>
__device__ __forceinline__ void rows_join(const qsa_paged_attn_args &a, const Joined &from, int x, int h0) {
    constexpr int D = 128 * S, LANES = D / 2;
    __shared__ float2 so[G > 1 ? JOIN_HEADS<S, G> : 1][G][LANES];
    __shared__ float sl[G > 1 ? JOIN_HEADS<S, G> : 1][G];
    const Work work(from.ws, from.cap, from.rows);
    const int tid = threadIdx.x, d = tid % LANES * 2, set = tid / LANES % G, in_block = tid / (LANES * G), h = h0 + in_block;
    const Part part = work.part[x];
    if (part.row < 0) return;
    const int n = h < from.rows ? part.n : 0;
    auto slot = [&](int p) { return ((size_t)(x + p * a.n_kv_heads) * 2 + (p == 0 ? 1 : 0)) * from.rows + h; };
    float top = -CUDART_INF_F, l = 0.0f;
#pragma unroll 4
    for (int p = 0; p < n; ++p) top = fmaxf(top, work.ml[slot(p) * 2]);
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int p = set; p < n; p += G) {
        const float2 ml = reinterpret_cast<const float2 *>(work.ml)[slot(p)];
        const float w = ml.x == -CUDART_INF_F ? 0.0f : exp2f(ml.x - top);
        l = fmaf(w, ml.y, l);
        o = __ffma2_rn(make_float2(w, w), *reinterpret_cast<const float2 *>(work.o + slot(p) * D + d), o);
    }
    if constexpr (G > 1) {
        so[in_block][set][d / 2] = o;
        if (d == 0) sl[in_block][set] = l;
        __syncthreads();
        if (set) return;
#pragma unroll
        for (int i = 1; i < G; ++i) {
            o = __fadd2_rn(o, so[in_block][i][d / 2]);
            l += sl[in_block][i];
        }
    }
    if (!n) return;
    const float inv = top == -CUDART_INF_F ? 0.0f : 1.0f / l;
    const size_t row = (size_t)part.row * a.n_q_heads + (size_t)(x % a.n_kv_heads) * from.rows + h;
    if (d == 0 && a.lse) a.lse[row] = lse_of(top, l);
    if (!QSA_IN(row * D + d + 1, (size_t)a.n_tokens * a.n_q_heads * D)) return;
    float2 y = make_float2(o.x * inv, o.y * inv);
    if (a.gate) {
        const float2 gate = __ldg(reinterpret_cast<const float2 *>(a.gate + row * D + d));
        y = make_float2(gated(y.x, gate.x), gated(y.y, gate.y));
    }
    store_out(a, row * D + d, y);
}
template <int S, int G>
__global__ void __launch_bounds__(JOIN_THREADS) paged_rows_join_kernel(const qsa_paged_attn_args a, const Joined from) {
    wait_for_previous_grid();
    allow_dependent_launch();
    rows_join<S, G>(a, from, blockIdx.x, blockIdx.y * (blockDim.x / (64 * S * G)));
}
template <int S>
cudaError_t launch_rows_join(const qsa_paged_attn_args &a, const Joined &from, cudaStream_t s) {
    if ((long long)a.n_tokens * a.n_kv_heads < 76)
        return launch_dependent(paged_rows_join_kernel<S, 4>, dim3(from.ctas, from.rows), dim3(256 * S), 0, s, a, from);
    const int heads = std::min(from.rows, JOIN_HEADS<S, 1>);
    return launch_dependent(paged_rows_join_kernel<S, 1>, dim3(from.ctas, (from.rows + heads - 1) / heads), dim3(64 * S * heads), 0, s, a, from);
}

// Whether rows of up to `cells` cells are shared out over CTAs, not taken whole: if the
// table can hold longer ones than WHOLE units, and there are fewer KV heads than CTAs
// (else there may also be more CTAs than the workspace has places for).
template <int S>
bool shared_out(const qsa_paged_attn_args &a, long long cells) {
    return cells > WHOLE * Shape<S>::UNIT && MAX_CTAS / a.n_kv_heads > 1;
}

// A call.  cells: the most that a row can go through.
template <int S, class A>
cudaError_t launch_rows(const A &a, long long cells, cudaStream_t s) {
    constexpr int UNIT = Shape<S>::UNIT;
    CUtensorMap kmap, vmap;
    cudaError_t e = encode<S>(kmap, a, a.kq);
    if (e == cudaSuccess) e = encode<S>(vmap, a, a.vq);
    if (e != cudaSuccess) return e;
    // A share per resident CTA; whole rows, and no join, where they are not shared out.
    const long long units = (cells + UNIT - 1) / UNIT;
    const int resident = std::max(MAX_CTAS / a.n_kv_heads, 1);
    const bool whole = !shared_out<S>(a, cells);
    const long long most = whole ? a.n_tokens : a.n_tokens * ((units + MIN_SHARE - 1) / MIN_SHARE);
    const int ranges = (int)std::min<long long>(most, resident), grid = ranges * a.n_kv_heads;
    const int per = a.n_q_heads / a.n_kv_heads;
    int block = 0;
    if constexpr (!LISTED<A> && !TREE<A>)
        block = !whole && may_take_groups<S>(a, units, group_block(per)) ? group_block(per) : 0;
    if (whole && units * UNIT <= SMALL && (long long)a.n_tokens * a.n_kv_heads > (units > 2 ? 2 : 1) * MAX_CTAS) {
        const int small = (int)std::min<long long>(a.n_tokens, std::max(152 * SMALL_PER_SM / a.n_kv_heads, 1));
        e = cudaFuncSetAttribute(paged_attn_kernel<S, 1, true, A>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<S, 1>));
        return e != cudaSuccess ? e
                                : launch_dependent(paged_attn_kernel<S, 1, true, A>, dim3(small * a.n_kv_heads), dim3(32), sizeof(Smem<S, 1>), s, a,
                                                   kmap, vmap, 0);
    }
    const auto kernel = whole ? paged_attn_kernel<S, NW, true, A> : paged_attn_kernel<S, NW, false, A>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<S, NW>));
    if (e == cudaSuccess) e = launch_dependent(kernel, dim3(grid), dim3(NW * 32), sizeof(Smem<S, NW>), s, a, kmap, vmap, block);
    if (e != cudaSuccess || whole) return e;
    if constexpr (LISTED<A> || TREE<A>)
        if (a.taken) return cudaSuccess;  // joined with the groups'
    if constexpr (LISTED<A> || TREE<A>) return launch_rows_join<S>(a, Joined{a.workspace, MAX_CTAS, per, grid}, s);
    const Joined one{a.workspace, MAX_CTAS, per, grid};
    Joined two{static_cast<uint8_t *>(a.workspace) + Work::bytes(MAX_CTAS, per, a.head_dim), MAX_GROUP_PARTS, GROUP_ROWS, 0};
    if constexpr (!LISTED<A> && !TREE<A>)
        if (block && (e = launch_paged_group(a, two.ws, two.ctas, s)) != cudaSuccess) return e;
    if (!block) two.rows = 0;
    return launch_join<S>(a, one, two, s);
}

}  // namespace
}  // namespace qsa
