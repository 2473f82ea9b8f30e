// qsa_page_score: what the keys of each page of a sequence can reach at most, by
// the page's bounds.
//
//   S = sum_d hi_d sum_heads max(q_d, 0) + lo_d sum_heads min(q_d, 0)
//
// The most that q . k can be for keys between lo and hi takes hi where q is
// positive and lo where it is negative; over heads that is linear in the sums of
// the positive and of the negative parts, so a page costs two rows of D codes and
// not one per head.  It is bound by reading the bounds, 2 D + 16 bytes per page
// and KV head, against 4 D flops per token.
//
// Pages are the M side (16 a warp) of m16n8k16 products, the sums of up to 4 NT
// tokens of one sequence the N side, as two fp16 parts each under a power of two
// per token (22 bits).  Codes go through shared memory (read straight to fragments,
// 32 bytes of a row at a time, the loads' tags took half of the time), a tile ahead.
// Lane (g, r) holds codes 8 S r .. 8 S r + 8 S - 1 of each quarter of pages g and g + 8,
// so that eight bytes (or sixteen) are one read and a k-step's dims are of one
// quarter; its products are summed per quarter, and the quarter's scale multiplies in
// fp32.
//
// The tiles of 16 pages of all sequences are shared out evenly over the blocks.  From
// 256 tokens on, where table rows are given, groups hold up to 32 tokens of one sequence,
// and a tile weighs what its group's tokens make it cost; by 32 tokens whatever they
// belong to, as a grid of tokens and tiles, 256 rows of one token took 207 us and 1984
// tokens of a prompt beside 60 such rows 514 where these take 38 and 69 (12 and 57 by
// themselves).  In us, 48/4 heads of 128, pages of 16, sequences of up to 32 K cells (of one
// token 8 K; without rows 24): 256 x 1 38, 64 x 4 31, 64 x 8 43, 32 x 16 28, 16 x 32 31.
//
// 61 tokens of 4 heads of 128 over pages of 16 of up to 32.7 K cells, 69 MB of bounds:
// 22.5 us, 3.1 TB/s (15.4 us from L2): issue 47 %, DRAM 37 %, latency of a warp's two
// tiles on their way.  One token over 469 pages: 4.1 us.  1984 tokens over 2 K pages of 16,
// 12/2 heads of 128: 57 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "check.cuh"
#include "page_share.cuh"
#include "qsa_internal.h"
#include "tc_common.cuh"

namespace qsa {
namespace {

constexpr int W = 4, THREADS = 32 * W;
constexpr int TILE = 16;  // pages of a warp at a time

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
// Codes 0 and 2 (or 1 and 3) of w.
__device__ __forceinline__ uint32_t pair(uint32_t w, bool odd) {
    return h2u(__hsub2(u2h(tc::prmt(w ^ 0x80808080u, 0x64646464u, odd ? 0x4341 : 0x4240)), u2h(0x64806480u)));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// The power of two that puts a token's largest sum into [2^13, 2^14), as far as
// it goes; 0 where that is 0, infinite or NaN.
__device__ __forceinline__ int sum_exponent(float m) {
    const uint32_t u = __float_as_uint(m);
    if (u == 0u || u >= 0x7F800000u) return 0;
    return min(max(13 - ((int)(u >> 23) - 127), -120), 120);
}

// What a tile of a group of n tokens costs: its codes' way to fragments, and products.
__device__ __forceinline__ int weight_of(int n) { return 4 + (n + 3) / 4; }

// The pages of token t's sequence.
__device__ __forceinline__ int pages_of(const qsa_page_score_args &a, int t, int &row, bool &bad) {
    row = a.rows ? __ldg(a.rows + t) : t;
    const int len = __ldg(a.seq_lens + t), most = a.max_pages * a.page_size;
    if (row < 0 || row >= a.n_rows) {
        bad = true;
        row = 0;
        return 0;
    }
    bad |= len < 0 || len > most;
    return (min(max(len, 0), most) + a.page_size - 1) >> (31 - __clz(a.page_size));
}

template <int S, int NT>
struct Smem {
    // The tokens' sums as B fragments: by bound, k-step, four tokens, lane.
    uint2 b[2][8 * S][NT][32];
    float unscale[4 * NT];      // 2^-e of a token
    int pages[4 * NT];
    uint32_t top[4 * NT];
    ShareSmem<W> found;
    // A warp's tiles: upper and lower bounds of sixteen pages.  Of many tokens one at a
    // time: their products hide the other warps' copies, and more blocks fit.
    static constexpr int STAGES = NT == 1 ? 2 : 1;
    alignas(16) uint8_t codes[W][STAGES][2][TILE * 128 * S];
    uint2 scales[W][STAGES][2][TILE];
};
// Place of 16-byte unit u of row r of a tile: the reads of a fragment meet a bank once.
template <int S>
__device__ __forceinline__ int unit_at(int r, int u) {
    return r * 128 * S + 16 * (S == 1 ? u ^ 2 * (r & 3) : u ^ 4 * (r & 1));
}
// Zeros where not `have`.
template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src, bool have) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(have ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(tc::smem_u32(dst)), "l"(src), "n"(BYTES), "r"(have ? BYTES : 0)
                     : "memory");
}

template <int S, int NT>
constexpr int CTAS_PER_SM = S == 1 ? (NT == 1 ? 5 : 3) : NT == 1 ? 3 : 2;  // by shared memory

// S = head_dim / 128.  A group: up to 4 NT consecutive tokens of one sequence, not
// across multiples of 4 NT; without rows, one token.
template <int S, int NT>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM<S, NT>) page_score_kernel(const qsa_page_score_args a) {
    constexpr int D = 128 * S, G = 4 * NT, Q = D / 4, KS = 2 * S;  // k-steps of a quarter
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<S, NT> &sh = *reinterpret_cast<Smem<S, NT> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, r = lane & 3;
    const int hkv = a.n_kv_heads, per = a.n_q_heads / hkv, kvh = blockIdx.x % hkv;
    const int range = blockIdx.x / hkv, ranges = gridDim.x / hkv;
    wait_for_previous_grid();
    allow_dependent_launch();
    bool bad = false;
    auto group_of = [&](int t, int &tiles) {  // by a warp: the group that starts at t, where one does
        const int u = t + lane;
        const bool same = u < min(a.n_tokens, t / G * G + G) && (lane == 0 || (a.rows && __ldg(a.rows + u) == __ldg(a.rows + t)));
        const unsigned m = __ballot_sync(0xffffffffu, same);
        const int n = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        int row;
        tiles = (__reduce_max_sync(0xffffffffu, lane < n ? pages_of(a, u, row, bad) : 0) + TILE - 1) / TILE;
        return n;
    };
    // This block's: tiles from i0 of the group that starts at t on; one token's, `left` in
    // all; else those up to the next share's, weights counted from the first token's.
    int t, i0, left = 0;
    long long total = 0, share = 0, pos = 0;  // all weights, a share's, those before t
    // The tile of the group of n tokens at `pos` with which share r starts, which starts in
    // it: the one whose weight does; a group whose sums cost more than its tiles weigh is
    // shared out evenly among as many shares as start in it, from its first tile on.
    auto split = [&](int r, int n, int tiles) {
        const long long w = weight_of(n), x = share * r;
        if (n <= 8) return (int)((x - pos + w - 1) / w);
        const int first = (int)((pos + share - 1) / share), m = (int)((pos + tiles * w + share - 1) / share) - first;
        return (int)((long long)(r - first) * tiles / m);
    };
    if constexpr (NT == 1) {
        auto tiles_of = [&](int t) {  // of the group that starts at t; 0 where none does
            int row, most = pages_of(a, t, row, bad);
            if (a.rows) {
                const int same = __ldg(a.rows + t);
                if (t % G && __ldg(a.rows + t - 1) == same) return 0;
#pragma unroll 1
                for (int u = t + 1; u < min(a.n_tokens, t / G * G + G) && __ldg(a.rows + u) == same; ++u) most = max(most, pages_of(a, u, row, bad));
            }
            return (most + TILE - 1) / TILE;
        };
        find_share(sh.found, a.n_tokens, range, ranges, 1, tiles_of, t, i0, left);
    } else {
        // Spans of 32 tokens, a quarter of them by each warp, a lane a token: the group that
        // starts there, if one does, weighs its tiles' weight.  All of them; then where the
        // share starts, by the warp that has it.  Not unrolled: it runs once.
        const int spans = (a.n_tokens + 31) / 32, run = (spans + W - 1) / W, s0 = min(warp * run, spans), s1 = min(s0 + run, spans);
        long long mine = 0, at = 0, x = 0;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            if (pass) {
                if (lane == 0) sh.found.part[warp] = mine;
                __syncthreads();
#pragma unroll 1
                for (int w = 0; w < W; ++w) {
                    at += w < warp ? sh.found.part[w] : 0;
                    total += sh.found.part[w];
                }
                share = max((total + ranges - 1) / ranges, 1ll);
                x = share * range;
                if (x < at || x >= at + mine) break;
            }
            int next_row = 0, next_pages = 0;
            auto load = [&](int s) {
                const int u = 32 * s + lane;
                next_row = next_pages = 0;
                if (s < s1 && u < a.n_tokens) {
                    int row;
                    next_row = __ldg(a.rows + u);
                    next_pages = pages_of(a, u, row, bad);
                }
            };
            load(s0);
#pragma unroll 1
            for (int s = s0; s < s1; ++s) {
                const int own = next_row, n = min(a.n_tokens - 32 * s, 32), before = __shfl_up_sync(0xffffffffu, own, 1);
                int most = next_pages, end = n;  // of the tokens from this one on; where its group ends
                load(s + 1);
                const unsigned starts = __ballot_sync(0xffffffffu, lane < n && (lane == 0 || own != before));
                if (starts == 1u) {
                    most = __reduce_max_sync(0xffffffffu, most);
                } else {
                    const unsigned later = starts & (0xfffffffeu << lane);
                    if (later) end = __ffs(later) - 1;
#pragma unroll 1
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_down_sync(0xffffffffu, most, o);
                        if (lane + o < end) most = max(most, v);
                    }
                }
                const int w = starts >> lane & 1u ? (most + TILE - 1) / TILE * weight_of(end - lane) : 0;
                const int all = __reduce_add_sync(0xffffffffu, w);
                if (!pass || x >= at + all) {
                    (pass ? at : mine) += all;
                    continue;
                }
                int upto = w;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                if (x >= at + upto - w && x < at + upto) {
                    sh.found.item = 32 * s + lane;
                    sh.found.before = at + upto - w;
                }
                break;
            }
        }
        __syncthreads();
        t = i0 = 0;
        pos = total;
        if (x < total) {
            t = sh.found.item;
            pos = sh.found.before;
            int tiles;
            const int n = group_of(t, tiles);
            i0 = split(range, n, tiles);
        }
    }
    while (t < a.n_tokens && (NT == 1 ? left > 0 : pos < total)) {
        int tiles;
        const int n = group_of(t, tiles), from = i0;
        const bool last = NT > 1 && share * (range + 1) < pos + (long long)tiles * weight_of(n);  // the share ends in this group
        const int i1 = NT == 1 ? min(tiles, i0 + left) : last ? split(range + 1, n, tiles) : tiles;
        if (i1 > from) {
            // The tokens' sums: a thread takes V dims of a token, of 32 tokens eight, so that a
            // token's are in one warp and the loads of all tokens are on their way together.
            constexpr int V = NT == 1 ? 2 : 8, LANES = D / V, AT_ONCE = THREADS / LANES, ROUNDS = (G + AT_ONCE - 1) / AT_ONCE;
            constexpr int AT_A_TIME = NT == 1 ? 8 : 8 / ROUNDS;  // heads whose loads are on their way together
            using Word = std::conditional_t<NT == 1, uint32_t, uint4>;
            __syncthreads();  // of the group before
            if (tid < G) {
                int row;
                sh.top[tid] = 0u;
                sh.pages[tid] = tid < n ? pages_of(a, t + tid, row, bad) : 0;
            }
            if constexpr (NT == 1) __syncthreads();
            const int d = tid % LANES * V, first = tid / LANES;
            float2 up[ROUNDS][V / 2], down[ROUNDS][V / 2];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i)
#pragma unroll
                for (int p = 0; p < V / 2; ++p) up[i][p] = down[i][p] = make_float2(0.0f, 0.0f);
            const size_t at = ((size_t)(t + first) * a.n_q_heads + (size_t)kvh * per) * D + d, next = (size_t)AT_ONCE * a.n_q_heads * D;
            auto load = [&](int i, int h) {
                const size_t from = at + i * next + (size_t)h * D;
                return first + i * AT_ONCE < n && h < per && QSA_IN(from + V - 1, (size_t)a.n_tokens * a.n_q_heads * D)
                           ? __ldg(reinterpret_cast<const Word *>(static_cast<const uint16_t *>(a.q) + from))
                           : Word{};
            };
            auto add = [&](int i, const Word &w) {
#pragma unroll
                for (int p = 0; p < V / 2; ++p) {
                    const uint32_t x = reinterpret_cast<const uint32_t *>(&w)[p];
                    const float2 v = a.dtype == QSA_F16 ? __half22float2(u2h(x))
                                                        : make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
                    up[i][p].x += fmaxf(v.x, 0.0f);
                    up[i][p].y += fmaxf(v.y, 0.0f);
                    down[i][p].x += fminf(v.x, 0.0f);
                    down[i][p].y += fminf(v.y, 0.0f);
                    // A NaN is lost in maximum and minimum.
                    if (v.x != v.x) up[i][p].x = v.x;
                    if (v.y != v.y) up[i][p].y = v.y;
                }
            };
            auto top_of = [&](int i) {
                float m = 0.0f;
#pragma unroll
                for (int p = 0; p < V / 2; ++p)
                    m = fmaxf(m, fmaxf(fmaxf(up[i][p].x, up[i][p].y), fmaxf(-down[i][p].x, -down[i][p].y)));
                return __float_as_uint(fabsf(m));  // not negative: bits order as values do
            };
            if constexpr (NT == 1) {
#pragma unroll
                for (int i = 0; i < ROUNDS; ++i) {
                    if (first + i * AT_ONCE >= n) continue;
#pragma unroll 1
                    for (int h = 0; h < per; h += AT_A_TIME) {
                        Word w[AT_A_TIME];
#pragma unroll
                        for (int e = 0; e < AT_A_TIME; ++e) w[e] = load(i, h + e);
#pragma unroll
                        for (int e = 0; e < AT_A_TIME; ++e) add(i, w[e]);
                    }
                    atomicMax(&sh.top[first + i * AT_ONCE], top_of(i));
                }
                __syncthreads();
            } else {
#pragma unroll 1
                for (int h = 0; h < per; h += AT_A_TIME) {
                    Word w[AT_A_TIME][ROUNDS];
#pragma unroll
                    for (int e = 0; e < AT_A_TIME; ++e)
#pragma unroll
                        for (int i = 0; i < ROUNDS; ++i) w[e][i] = load(i, h + e);
#pragma unroll
                    for (int i = 0; i < ROUNDS; ++i) {
                        if (i * AT_ONCE >= n) break;
#pragma unroll
                        for (int e = 0; e < AT_A_TIME; ++e) add(i, w[e][i]);
                    }
                }
            }
            __half *frag = reinterpret_cast<__half *>(sh.b);
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int k = first + i * AT_ONCE;
                uint32_t top;
                if constexpr (NT == 1) {
                    top = sh.top[k];
                } else {
                    top = top_of(i);
#pragma unroll
                    for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                }
                if (k >= (n + 3) / 4 * 4) continue;  // no product takes them
                const int ex = sum_exponent(__uint_as_float(top));
                const float f = exp2i(ex);
                if (tid % LANES == 0) sh.unscale[k] = exp2i(-ex);
#pragma unroll
                for (int p = 0; p < V / 2; ++p) {
                    // Place of dims d + 2 p and the next (of different halves of a k-step) as codes of a quarter.
                    const int in = (d + 2 * p) % Q, rr = in / (8 * S), e = in % (8 * S), ks = d / Q * KS + e / 4;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float2 v = b ? down[i][p] : up[i][p];
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            // Beside an infinite sum the finite ones, which have no power of two
                            // then, count for nothing.
                            float x = (odd ? v.y : v.x) * f;
                            if (top >= 0x7F800000u && fabsf(x) < CUDART_INF_F) x = 0.0f;
                            const __half hi = __float2half_rn(x), lo = fabsf(x) < CUDART_INF_F ? __float2half_rn(x - __half2float(hi)) : __half(0.0f);
                            // Column 2 (k % 4) + part, row: register `odd`, half by the pair.
                            const size_t at = ((((size_t)b * 8 * S + ks) * NT + k / 4) * 32 + (2 * (k % 4)) * 4 + rr) * 4 + odd * 2 + (e % 4) / 2;
                            frag[at] = hi;
                            frag[at + 16] = lo;
                        }
                    }
                }
            }
            __syncthreads();
            int row;
            pages_of(a, t, row, bad);
            const int most = tiles * TILE;  // pages of the longest token, or a few more
            // The warp's tiles, one ahead of the products and its pages one more: 16-byte
            // units of a page's row next to one another, eight lanes (or sixteen) a row.
            int page = -1;  // of row lane % 16
            auto look = [&](int i) {
                const int j = i * TILE + (lane & 15);
                page = i < i1 && j < a.max_pages && j < most ? __ldg(a.page_table + (size_t)row * a.max_pages + j) : -1;
            };
            unsigned held = 0u;  // rows that are there: sixteen of the tile at hand, sixteen of the next
            auto copy = [&](int st) {
                bool there = page >= 0 && page < a.n_pages;
                const size_t at = (size_t)(there ? page : 0) * hkv + kvh;
                there = there && QSA_IN(at, (size_t)a.n_pages * hkv);
                const unsigned m = __ballot_sync(0xffffffffu, there);
                held = held >> 16 | m << 16;
                cp_async<8>(&sh.scales[warp][st][lane >> 4][lane & 15], (lane >> 4 ? a.lo_sc : a.hi_sc) + at * 4, there);
                constexpr int UNITS = 8 * S, ROWS = 32 / UNITS;  // of a row; rows at a time
                const int u = lane % UNITS;
#pragma unroll
                for (int x = 0; x < TILE / ROWS; ++x) {
                    const int r16 = x * ROWS + lane / UNITS;
                    const size_t from = (size_t)__shfl_sync(0xffffffffu, (unsigned long long)at, r16) * D + 16 * u;
                    uint8_t *to = sh.codes[warp][st][0] + unit_at<S>(r16, u);
                    cp_async<16>(to, a.hi_q + from, m >> r16 & 1u);
                    cp_async<16>(to + TILE * D, a.lo_q + from, m >> r16 & 1u);
                }
                asm volatile("cp.async.commit_group;\n" ::);
            };
            constexpr int STAGES = Smem<S, NT>::STAGES;
            int st = 0;
            look(from + warp);
            copy(0);
            look(from + warp + W);
            for (int i = from + warp; i < i1; i += W, st ^= STAGES - 1) {
                if constexpr (STAGES == 2) {
                    copy(st ^ 1);
                    look(i + 2 * W);
                    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
                } else {
                    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
                }
                __syncwarp();
                const unsigned held_now = STAGES == 2 ? held : held >> 16;
                const bool there[2] = {(held_now >> g & 1u) != 0u, (held_now >> (g + 8) & 1u) != 0u};
                auto products = [&](auto columns) {  // with the sums of the first 4 K tokens
                    constexpr int K = decltype(columns)::value;
                    float y[K][4];
#pragma unroll
                    for (int k = 0; k < K; ++k) y[k][0] = y[k][1] = y[k][2] = y[k][3] = 0.0f;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint2 sc[2] = {sh.scales[warp][st][b][g], sh.scales[warp][st][b][g + 8]};
                        const uint8_t *codes = sh.codes[warp][st][b];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float s[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const __half2 h = u2h(q >> 1 ? sc[e].y : sc[e].x);
                                s[e] = q & 1 ? __high2float(h) : __low2float(h);
                            }
                            uint32_t w[2][2 * S];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if constexpr (S == 1)
                                    *reinterpret_cast<uint2 *>(w[e]) = *reinterpret_cast<const uint2 *>(codes + unit_at<S>(g + 8 * e, 2 * q + (r >> 1)) + 8 * (r & 1));
                                else
                                    *reinterpret_cast<uint4 *>(w[e]) = *reinterpret_cast<const uint4 *>(codes + unit_at<S>(g + 8 * e, 4 * q + r));
                            }
                            uint32_t x[KS][4];
#pragma unroll
                            for (int c = 0; c < KS; ++c) {
                                x[c][0] = pair(w[0][c], false);
                                x[c][1] = pair(w[1][c], false);
                                x[c][2] = pair(w[0][c], true);
                                x[c][3] = pair(w[1][c], true);
                            }
#pragma unroll
                            for (int k = 0; k < K; ++k) {
                                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                for (int c = 0; c < KS; ++c) mma(acc, x[c], sh.b[b][q * KS + c][k][lane]);
                                y[k][0] = fmaf(acc[0] + acc[1], s[0], y[k][0]);
                                y[k][2] = fmaf(acc[2] + acc[3], s[1], y[k][2]);
                            }
                        }
                    }
                    __syncwarp();  // the tile has been read
                    if constexpr (STAGES == 1) {
                        copy(0);
                        look(i + 2 * W);
                    }
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const int token = 4 * k + r;
                        if (token >= n) continue;
                        const int count = sh.pages[token];
                        const float f = sh.unscale[token];
                        float *dst = a.scores + ((size_t)(t + token) * hkv + kvh) * a.ld;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = i * TILE + g + 8 * e;
                            if (j >= count) continue;
                            bad |= !there[e];
                            if (QSA_IN(((size_t)(t + token) * hkv + kvh) * a.ld + j, (size_t)a.n_tokens * hkv * a.ld))
                                dst[j] = there[e] ? y[k][2 * e] * f : -CUDART_INF_F;
                        }
                    }
                };
                if (NT == 1 || n <= 4)
                    products(std::integral_constant<int, 1>{});
                else if (n <= 16)
                    products(std::integral_constant<int, NT == 1 ? 1 : 4>{});
                else
                    products(std::integral_constant<int, NT>{});
            }
        }
        asm volatile("cp.async.wait_group 0;\n" ::: "memory");
        __syncwarp();
        if (last) break;
        if constexpr (NT == 1) left -= i1 - from;
        pos += (long long)tiles * weight_of(n);
        i0 = 0;
        t += max(n, 1);
    }
    if (__syncthreads_or(bad) && tid == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
}

template <int S, int NT>
cudaError_t launch(const qsa_page_score_args &a, cudaStream_t s) {
    constexpr int SMEM = (int)sizeof(Smem<S, NT>);
    cudaError_t e = cudaFuncSetAttribute(page_score_kernel<S, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    const long long tiles = (a.max_pages + TILE - 1) / TILE;
    const int ranges = (int)std::min<long long>(a.n_tokens * tiles, std::max(152 * CTAS_PER_SM<S, NT> / a.n_kv_heads, 1));
    return launch_dependent(page_score_kernel<S, NT>, dim3(ranges * a.n_kv_heads), dim3(THREADS), SMEM, s, a);
}

}  // namespace

cudaError_t launch_page_score(const qsa_page_score_args &a, cudaStream_t s) {
    const bool many = a.rows && a.n_tokens >= 256;
    if (a.head_dim == 128) return many ? launch<1, 8>(a, s) : launch<1, 1>(a, s);
    return many ? launch<2, 8>(a, s) : launch<2, 1>(a, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_page_score)
