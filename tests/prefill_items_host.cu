// Walks the prefill kernels' work items on the host. stdin: lines of "G mbps T max_q
// window sinks R  context_lens[R]  query_start[R + 1]"; prints per line the items,
// those that leave q's rows or a table's columns, and the rows of q counted once per
// KV head by the plain tiles and by the sliding ones.
#include <cstdio>
#include <vector>

#include "prefill_items.cuh"

using namespace mi;

int main() {
    int G, mbps, T, max_q, window, sinks, R;
    while (std::scanf("%d %d %d %d %d %d %d", &G, &mbps, &T, &max_q, &window, &sinks, &R) == 7) {
        std::vector<int32_t> lens(R), start(R + 1);
        for (int32_t& x : lens)
            if (std::scanf("%d", &x) != 1) return 1;
        for (int32_t& x : start)
            if (std::scanf("%d", &x) != 1) return 1;
        const PrefillBatch p = {lens.data(), start.data(), G, mbps, T, max_q};
        const int cap = mbps * kBlock;
        long long items = 0, bad = 0, rows = 0, slide_rows = 0;
        for (int r = 0; r < R; ++r) {
            for (int tile_rows : {64, 128 / G * G, 2 * (128 / G * G)}) {
                Item it;
                for (int k = 0; tile_item(p, tile_rows, r, k, it); ++k) {
                    ++items;
                    const long long q1 = it.q0 + (long long)it.m;
                    bad += it.q0 < 0 || it.m < 1 || q1 > T || it.rho0 < 0 || it.rows_here < 1 ||
                           it.rho0 + (long long)it.rows_here > (long long)it.m * G || it.n < 0 || it.n > cap ||
                           it.first < -it.m || it.p_hi >= it.n || it.nblk < 0 || it.nblk > mbps;
                    if (tile_rows == 64) rows += it.rows_here;
                }
            }
            const int item_rows = 2 * (128 / G * G), tiles = slide_tiles(p, r, item_rows);
            for (int k = 0; k < tiles; ++k) {
                const SlideItem it = slide_tile_item(p, window, sinks, item_rows, r, 0, tiles, k);
                ++items;
                const long long q1 = it.q0 + (long long)it.m;
                bad += it.q0 < 0 || it.m < 1 || q1 > T || it.tok0 < 0 || it.tok0 >= it.m || it.n < 0 || it.n > cap ||
                       it.first < -it.m || it.p_hi >= it.n || it.nblk < 0 || it.gap < 0 || it.head < 0 ||
                       (long long)it.nblk + it.gap > mbps || it.lo < 0 || it.sinks < 0 || it.sinks > it.lo;
                slide_rows += (long long)(it.tok0 + item_rows / G < it.m ? item_rows / G : it.m - it.tok0) * G;
            }
        }
        std::printf("%lld %lld %lld %lld\n", items, bad, rows, slide_rows);
    }
    return 0;
}
