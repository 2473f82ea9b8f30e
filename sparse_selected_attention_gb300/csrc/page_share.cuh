// How a block finds its share of work that is a number of pieces for each of some
// items (tokens, rows), when only the device knows the numbers: all blocks count for
// themselves, which costs less than a launch before them.  The loops are not
// unrolled: it runs once, and an instruction's first fetch costs more than its
// execution.
#pragma once

namespace qsa {
namespace {

template <int W>
struct ShareSmem {
    long long part[W], before;
    int item;
};

// Block `range` of `ranges` gets `left` pieces from piece `first` of `item` on; 0:
// none.  count(i): item i's.  least: of a share.  All threads of W warps call it.
template <int W, class F>
__device__ __forceinline__ void find_share(ShareSmem<W> &sh, int n, int range, int ranges, int least, F &&count, int &item, int &first, int &left) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long total = 0, done = 0, x = 0;
    int share = 0;
    const bool once = n <= 32 * W;
#pragma unroll 1
    for (int pass = 0; pass < (once ? 1 : 2); ++pass) {  // all pieces; then where the share starts
        done = 0;
#pragma unroll 1
        for (int base = 0; base < n; base += 32 * W) {
            const int c = base + tid < n ? count(base + tid) : 0;
            long long sum = c;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (lane == 31) sh.part[warp] = sum;
            __syncthreads();
            long long before = done + sum - c, all = 0;
#pragma unroll 1
            for (int w = 0; w < W; ++w) {
                const long long v = sh.part[w];
                before += w < warp ? v : 0;
                all += v;
            }
            done += all;
            if (!pass) total = done;
            if (pass || once) {
                share = (int)max((total + ranges - 1) / ranges, (long long)least);
                x = (long long)share * range;
                if (c && x >= before && x < before + c) {
                    sh.item = base + tid;
                    sh.before = before;
                }
            }
            __syncthreads();
        }
    }
    left = (int)max(min((long long)share, total - x), 0ll);
    item = left ? sh.item : 0;
    first = left ? (int)(x - sh.before) : 0;
}

}  // namespace
}  // namespace qsa
