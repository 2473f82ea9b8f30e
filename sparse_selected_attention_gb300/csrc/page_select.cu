// qsa_page_select: for each token and KV head the first pages, the last ones and
// the best-scoring others up to a budget, in order.
//
// Scores become keys that order as they do (a NaN lowest).  The k-th largest key of
// the pages to choose from is found by counting: the keys between the smallest and
// the largest go to up to 512 bins by their leading bits, the bin that the k-th is in
// is the next range, and so on until its keys are few enough to be compared with one
// another (of scores that are no odd lot the first range's, mostly).  Pages above the
// key are taken, and the lowest-numbered of those equal to it.
//
// It would be bound by reading the scores once; what it takes is the chain of counts
// and exchanges of a row, which other rows on the SM hide: 128 of 1875 to 2000 pages for
// 3968 rows, 31 MB, 22.6 us, 1.4 TB/s at 70 % of the issue slots (51 us by finding the key
// bit by bit); 32 of 469 for one, 2.9 us.  A block takes one token
// and head.  Its warps hold runs of consecutive pages in registers, so that a warp's
// pages are read in whole lines, and a word of bits per 32 pages is listed by a lane.
#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

// Never 0, which stands for a page that is not to be chosen from.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is +0
    return x != x ? 1u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int BINS = 512, FEW = 64;  // keys that are compared with one another

template <int W>
struct SelectSmem {
    alignas(16) int bins[BINS];
    uint32_t few[FEW];
    int n_few;
    uint32_t low[W], high[W], least_high[W];
    int sure[W], equal[W];
    // What warp 0 found: the next range, the keys above it, those still wanted from
    // it, and those in it.
    uint32_t lo, hi;
    int above, need, count;
};

template <int W>
__device__ __forceinline__ void row_sync() {
    if constexpr (W == 1)
        __syncwarp();
    else
        __syncthreads();
}

// KEYS: pages a lane holds in registers; 0: a row's scores are read again (from L2)
// for each step.
template <int W, int KEYS>
__global__ void __launch_bounds__(32 * W) page_select_kernel(const qsa_page_select_args a) {
    constexpr bool HELD = KEYS > 0;
    __shared__ SelectSmem<W> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long item = blockIdx.x;
    const int t = (int)(item / a.n_kv_heads);
    wait_for_previous_grid();
    allow_dependent_launch();
    const int len = __ldg(a.seq_lens + t), shift = 31 - __clz(a.page_size);
    const long long pages = len <= 0 ? 0 : ((long long)len + a.page_size - 1) >> shift;
    if ((len < 0 || pages > a.ld) && tid == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
    const int n = (int)min(pages, (long long)a.ld), take = min(n, a.budget);
    int32_t *out = a.pages + item * a.width;
    const float *scores = a.scores + item * a.ld;
    const bool in = QSA_IN(item * a.width + a.width - 1, (long long)a.n_tokens * a.n_kv_heads * a.width) &&
                    QSA_IN(item * a.ld + n - (n > 0), (long long)a.n_tokens * a.n_kv_heads * a.ld);
    if (!in) return;
    if (tid == 0) a.counts[item] = take;
    for (int i = (n <= a.budget ? 0 : take) + tid; i < a.width; i += 32 * W) out[i] = i < take ? i : -1;
    if (n <= a.budget) return;
    // The free pages sink .. last-1; `want` of them are chosen.
    const int sink = a.sink, last = n - a.local, want = take - sink - a.local;
    // This warp's run of pages, whole lanes of 32.
    const int steps = ((n + 31) / 32 + W - 1) / W, base = warp * steps * 32;
    auto is_free = [&](int i) {
        const int p = base + 32 * i + lane;
        return p >= sink && p < last;
    };
    auto load = [&](int i) -> uint32_t { return is_free(i) ? key_of(__ldg(scores + base + 32 * i + lane)) : 0u; };
    uint32_t held[HELD ? KEYS : 1];
    if constexpr (HELD) {
        float x[KEYS];
#pragma unroll
        for (int i = 0; i < KEYS; ++i) x[i] = i < steps && is_free(i) ? __ldg(scores + base + 32 * i + lane) : 0.0f;
#pragma unroll
        for (int i = 0; i < KEYS; ++i) held[i] = i < steps && is_free(i) ? key_of(x[i]) : 0u;
    }
    auto each = [&](auto &&f) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i) f(i, held[i]);
        } else {
            constexpr int BATCH = 8;  // loads on their way
            for (int i = 0; i < steps; i += BATCH) {
                uint32_t k[BATCH];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) k[j] = i + j < steps ? load(i + j) : 0u;
#pragma unroll
                for (int j = 0; j < BATCH; ++j)
                    if (i + j < steps) f(i + j, k[j]);
            }
        }
    };
    uint32_t cut = 0xffffffffu;  // keys above it are chosen, and `ties` of those equal to it
    int ties = 0;
    if (want > 0) {
        // From the least of the threads' largest keys on there is one key a thread: as
        // low as the range has to go if that is enough (of 16 keys a thread it leaves
        // three quarters of them out).  Else, from the least key.
        uint32_t lo = 0xffffffffu, hi = 0u;
        each([&](int, uint32_t k) {
            lo = min(lo, k - 1);
            hi = max(hi, k);
        });
        uint32_t least_hi = __reduce_min_sync(0xffffffffu, hi);
        lo = __reduce_min_sync(0xffffffffu, lo) + 1;
        hi = __reduce_max_sync(0xffffffffu, hi);
        if constexpr (W > 1) {
            if (lane == 0) {
                sh.low[warp] = lo;
                sh.high[warp] = hi;
                sh.least_high[warp] = least_hi;
            }
        }
        for (int i = tid; i < BINS; i += 32 * W) sh.bins[i] = 0;
        if (tid == 0) sh.n_few = 0;
        row_sync<W>();
        if constexpr (W > 1) {
            lo = __reduce_min_sync(0xffffffffu, lane < W ? sh.low[lane] - 1 : 0xffffffffu) + 1;  // 0: no key in the warp
            hi = __reduce_max_sync(0xffffffffu, lane < W ? sh.high[lane] : 0u);
            least_hi = __reduce_min_sync(0xffffffffu, lane < W ? sh.least_high[lane] : 0xffffffffu);
        }
        if (least_hi > 0u && want <= 32 * W) lo = least_hi;
        int need = want;
        while (lo < hi) {  // of the keys in lo .. hi the need-th largest is the cut; the bins are 0
            const int drop = max(32 - __clz(hi - lo) - 9, 0);
            each([&](int, uint32_t k) {
                if (k - lo <= hi - lo) atomicAdd(&sh.bins[(k - lo) >> drop], 1);
            });
            row_sync<W>();
            if (warp == 0) {
                // Sixteen bins a lane, the lanes from the top.
                const int top = BINS - 1 - 16 * lane;
                int mine = 0;
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const int4 v = *reinterpret_cast<const int4 *>(&sh.bins[top - 15 + i]);
                    mine += v.x + v.y + v.z + v.w;
                }
                int upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                if (upto >= need && upto - mine < need) {
                    int before = upto - mine, b = top;
                    while (before + sh.bins[b] < need) before += sh.bins[b--];
                    sh.need = need - before;
                    sh.count = sh.bins[b];
                    sh.lo = lo + ((uint32_t)b << drop);
                    sh.hi = min(hi, sh.lo + (1u << drop) - 1);
                }
            }
            row_sync<W>();
            lo = sh.lo;
            hi = sh.hi;
            need = sh.need;
            const int count = sh.count;
            if (count <= FEW) {
                if (lo < hi) {
                    each([&](int, uint32_t k) {
                        if (k - lo <= hi - lo) sh.few[atomicAdd(&sh.n_few, 1)] = k;
                    });
                    row_sync<W>();
                    for (int mine = tid; mine < count; mine += 32 * W) {
                        const uint32_t k = sh.few[mine];
                        int more = 0, same = 0;
                        for (int i = 0; i < count; ++i) {
                            more += sh.few[i] > k;
                            same += sh.few[i] == k;
                        }
                        if (more < need && more + same >= need) {  // the same in all threads that find it so
                            sh.lo = k;
                            sh.above = more;
                        }
                    }
                    row_sync<W>();
                    lo = hi = sh.lo;
                    need -= sh.above;
                }
                break;
            }
            for (int i = tid; i < BINS; i += 32 * W) sh.bins[i] = 0;
            row_sync<W>();
        }
        cut = lo;
        ties = need;
    }
    if constexpr (HELD) {
        // A word of chosen pages and one of pages at the cut for each 32 of them, lane i
        // the warp's i-th.
        uint32_t mine_sure = 0u, mine_equal = 0u;
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const bool forced = held[i] == 0u && i < steps && base + 32 * i + lane < n;
            const uint32_t sure = __ballot_sync(0xffffffffu, forced || held[i] > cut);
            const uint32_t equal = __ballot_sync(0xffffffffu, held[i] == cut);
            if (lane == i) {
                mine_sure = sure;
                mine_equal = equal;
            }
        }
        // Before this lane's word: pages at the cut, of which the first `ties` are chosen.
        const int n_equal = __popc(mine_equal), n_sure = __popc(mine_sure);
        int equal = n_equal, sure = n_sure;
#pragma unroll
        for (int o = 1; o < KEYS; o <<= 1) {
            const int e = __shfl_up_sync(0xffffffffu, equal, o), s = __shfl_up_sync(0xffffffffu, sure, o);
            if (lane >= o) {
                equal += e;
                sure += s;
            }
        }
        if constexpr (W > 1) {
            if (lane == KEYS - 1) {
                sh.equal[warp] = equal;
                sh.sure[warp] = sure;
            }
            __syncthreads();
            equal += __reduce_add_sync(0xffffffffu, lane < warp ? sh.equal[lane] : 0);
            sure += __reduce_add_sync(0xffffffffu, lane < warp ? sh.sure[lane] : 0);
        }
        equal -= n_equal;
        sure -= n_sure;
        int at = sure + min(equal, ties), left = ties - equal;
        uint32_t word = mine_sure;
        for (uint32_t e = mine_equal; e && left > 0; e &= e - 1, --left) word |= e & -e;
        for (int first = base + 32 * lane; word; word &= word - 1) out[at++] = first + __ffs(word) - 1;
    } else {
        int sure = 0, equal = 0;
        each([&](int i, uint32_t k) {
            const int p = base + 32 * i + lane;
            sure += __popc(__ballot_sync(0xffffffffu, p < n && (k == 0u || k > cut)));
            equal += __popc(__ballot_sync(0xffffffffu, k == cut));
        });
        if (lane == 0) {
            sh.sure[warp] = sure;
            sh.equal[warp] = equal;
        }
        __syncthreads();
        int sure_before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.sure[lane] : 0);
        int equal_before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.equal[lane] : 0);
        const unsigned under = (1u << lane) - 1;
        each([&](int i, uint32_t k) {
            const int p = base + 32 * i + lane;
            const bool yes = p < n && (k == 0u || k > cut), tie = k == cut;
            const unsigned sures = __ballot_sync(0xffffffffu, yes), equals = __ballot_sync(0xffffffffu, tie);
            const int e = equal_before + __popc(equals & under), at = sure_before + __popc(sures & under) + min(e, ties);
            if (yes || (tie && e < ties)) out[at] = p;
            sure_before += __popc(sures);
            equal_before += __popc(equals);
        });
    }
}

template <int W, int KEYS>
cudaError_t launch(const qsa_page_select_args &a, cudaStream_t s) {
    return launch_dependent(page_select_kernel<W, KEYS>, dim3((unsigned)((long long)a.n_tokens * a.n_kv_heads)), dim3(32 * W), 0, s, a);
}

}  // namespace

// Few rows: many threads and few keys each, for the latency.  Many: enough keys a
// thread that a row's fixed part does not count.  us, by threads x keys:
//   1 row of 469 pages      256 x 2 2.7, 128 x 4 3.1, 128 x 16 3.8
//   1984 rows of 469        256 x 2 8.0, 128 x 4 6.6, 128 x 8 7.9
//   256 rows of 2000        256 x 8 4.3, 128 x 16 5.0, 512 x 4 4.4
//   3968 rows of 1999       256 x 8 24.4, 128 x 16 21.5, 512 x 4 31.9
//   1000 rows of 4000       512 x 8 14.2, 256 x 16 12.7; 1 row 3.9, 4.8
cudaError_t launch_page_select(const qsa_page_select_args &a, cudaStream_t s) {
    const bool few = (long long)a.n_tokens * a.n_kv_heads <= 152 * 4;
    if (a.ld <= 512) return few ? launch<8, 2>(a, s) : launch<4, 4>(a, s);
    if (a.ld <= 2048) return few ? launch<8, 8>(a, s) : launch<4, 16>(a, s);
    if (a.ld <= 4096) return few ? launch<16, 8>(a, s) : launch<8, 16>(a, s);
    if (a.ld <= 16384) return launch<32, 16>(a, s);
    return launch<32, 0>(a, s);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_page_select)
