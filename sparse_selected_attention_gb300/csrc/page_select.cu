// qsa_page_select: for each token and KV head the first pages, the last ones and
// the best-scoring others up to a budget, in order.
//
// Scores become keys that order as they do (a NaN lowest), and the k-th largest
// key of the pages to choose from is found by halving the range between the
// smallest and the largest: a step counts the keys from its middle on, and ends
// the search where they are k.  Pages above it are taken, and the lowest-numbered
// of those equal to it.
//
// A block takes one token and head.  Its warps hold runs of consecutive pages, so
// that a warp's pages are read in whole lines and listed by counting.
#include "check.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

// Pages in registers: KEYS a lane.  A longer row's scores are read again (from
// L2) for each step.
constexpr int KEYS = 16;

__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is +0
    return x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int W, bool HELD>
__global__ void __launch_bounds__(32 * W) page_select_kernel(const qsa_page_select_args a) {
    __shared__ int found[2][2][W];
    __shared__ uint32_t range[2][W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long item = blockIdx.x;
    const int t = (int)(item / a.n_kv_heads);
    wait_for_previous_grid();
    allow_dependent_launch();
    const int len = __ldg(a.seq_lens + t), shift = 31 - __clz(a.page_size);
    long long pages = len <= 0 ? 0 : ((long long)len + a.page_size - 1) >> shift;
    if ((len < 0 || pages > a.ld) && threadIdx.x == 0 && a.err) atomicOr(a.err, QSA_DEVERR_BAD_ID);
    const int n = (int)min(pages, (long long)a.ld), take = min(n, a.budget);
    int32_t *out = a.pages + item * a.width;
    const float *scores = a.scores + item * a.ld;
    if (threadIdx.x == 0) a.counts[item] = take;
    if (n <= a.budget) {
        for (int i = threadIdx.x; i < a.width; i += 32 * W)
            if (QSA_IN(item * a.width + i, (long long)a.n_tokens * a.n_kv_heads * a.width)) out[i] = i < n ? i : -1;
        return;
    }
    // The free pages sink .. last-1; `want` of them are chosen.
    const int sink = a.sink, last = n - a.local, want = take - sink - a.local;
    // This warp's run of pages, whole lanes of 32.
    const int steps = ((n + 31) / 32 + W - 1) / W, base = warp * steps * 32;
    uint32_t held[HELD ? KEYS : 1];
    auto load = [&](int i) -> uint32_t {  // of the lane's i-th page; 0 where it is not free
        const int p = base + 32 * i + lane;
        return p >= sink && p < last && QSA_IN(item * a.ld + p, (long long)a.n_tokens * a.n_kv_heads * a.ld) ? key_of(__ldg(scores + p)) : 0u;
    };
    auto is_free = [&](int i) {
        const int p = base + 32 * i + lane;
        return p >= sink && p < last;
    };
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < KEYS; ++i) held[i] = i < steps ? load(i) : 0u;
    }
    auto each = [&](auto &&f) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i)
                if (i < steps) f(i, held[i]);
        } else {
            for (int i = 0; i < steps; ++i) f(i, load(i));
        }
    };
    int turn = 0;
    auto block_sum = [&](int x) {  // of the warps' values
        if constexpr (W == 1) return x;
        turn ^= 1;
        if (lane == 0) found[0][turn][warp] = x;
        __syncthreads();
        int v = lane < W ? found[0][turn][lane] : 0;
        return __reduce_add_sync(0xffffffffu, v);
    };
    uint32_t cut = 0xffffffffu;  // the least key that is chosen, and how many lie above it
    int above = 0;
    if (want > 0) {
        uint32_t lo = 0xffffffffu, hi = 0u;
        each([&](int i, uint32_t k) {
            if (is_free(i)) {
                lo = min(lo, k);
                hi = max(hi, k);
            }
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if constexpr (W > 1) {
            if (lane == 0) {
                range[0][warp] = lo;
                range[1][warp] = hi;
            }
            __syncthreads();
            lo = __reduce_min_sync(0xffffffffu, lane < W ? range[0][lane] : 0xffffffffu);
            hi = __reduce_max_sync(0xffffffffu, lane < W ? range[1][lane] : 0u);
        }
        // At least `want` keys are from lo on, and fewer from hi + 1 on.
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            int c = 0;
            each([&](int, uint32_t k) { c += k >= mid; });  // mid > lo >= 0: pages that are not free do not count
            c = block_sum(__reduce_add_sync(0xffffffffu, c));
            if (c >= want) {
                lo = mid;
                if (c == want) break;
            } else {
                hi = mid - 1;
            }
        }
        cut = lo;
        int c = 0;
        each([&](int i, uint32_t k) { c += is_free(i) && k > cut; });
        above = block_sum(__reduce_add_sync(0xffffffffu, c));
    }
    const int ties = want - above;  // of the pages at the cut, the lowest-numbered
    int sure = 0, equal = 0;
    each([&](int i, uint32_t k) {
        const int p = base + 32 * i + lane;
        const bool free = is_free(i), yes = p < n && (!free || (want > 0 && k > cut));
        sure += __popc(__ballot_sync(0xffffffffu, yes));
        equal += __popc(__ballot_sync(0xffffffffu, free && want > 0 && k == cut));
    });
    int sure_before = 0, equal_before = 0;
    if constexpr (W > 1) {
        __syncthreads();
        if (lane == 0) {
            found[0][0][warp] = sure;
            found[1][0][warp] = equal;
        }
        __syncthreads();
        sure_before = __reduce_add_sync(0xffffffffu, lane < warp ? found[0][0][lane] : 0);
        equal_before = __reduce_add_sync(0xffffffffu, lane < warp ? found[1][0][lane] : 0);
    }
    const unsigned under = (1u << lane) - 1;
    each([&](int i, uint32_t k) {
        const int p = base + 32 * i + lane;
        const bool free = is_free(i), yes = p < n && (!free || (want > 0 && k > cut)), tie = free && want > 0 && k == cut;
        const unsigned sures = __ballot_sync(0xffffffffu, yes), equals = __ballot_sync(0xffffffffu, tie);
        const int e = equal_before + __popc(equals & under), at = sure_before + __popc(sures & under) + min(e, ties);
        if ((yes || (tie && e < ties)) && QSA_IN(item * a.width + at, (long long)a.n_tokens * a.n_kv_heads * a.width)) out[at] = p;
        sure_before += __popc(sures);
        equal_before += __popc(equals);
    });
    for (int i = take + threadIdx.x; i < a.width; i += 32 * W)
        if (QSA_IN(item * a.width + i, (long long)a.n_tokens * a.n_kv_heads * a.width)) out[i] = -1;
}

}  // namespace

cudaError_t launch_page_select(const qsa_page_select_args &a, cudaStream_t s) {
    const dim3 grid((unsigned)((long long)a.n_tokens * a.n_kv_heads));
    if (a.ld <= 32 * KEYS) return launch_dependent(page_select_kernel<1, true>, grid, dim3(32), 0, s, a);
    if (a.ld <= 4 * 32 * KEYS) return launch_dependent(page_select_kernel<4, true>, grid, dim3(128), 0, s, a);
    if (a.ld <= 32 * 32 * KEYS) return launch_dependent(page_select_kernel<32, true>, grid, dim3(1024), 0, s, a);
    return launch_dependent(page_select_kernel<32, false>, grid, dim3(1024), 0, s, a);
}

}  // namespace qsa

QSA_DEFINE_CHECK_READER(take_check_word_page_select)
