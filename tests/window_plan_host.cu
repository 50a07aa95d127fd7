// Walks the plan of mi_paged_prefill_scores on the host: which slots of partial
// log-sum-exps the first launch writes, and which ones the later launches read.
// stdin: lines of "Hkv G R max_q grid resident  n m  n m ..."; prints per line
// the slots the workspace has, written, the largest slot read and the reads of
// slots that were not written.
#include <cstdio>
#include <vector>

#include "window.cuh"

using namespace mi;
using namespace mi::window;

int main() {
    int Hkv, G, R, max_q, grid, resident;
    while (std::scanf("%d %d %d %d %d %d", &Hkv, &G, &R, &max_q, &grid, &resident) == 6) {
        std::vector<int32_t> lens(R), start(R + 1, 0);
        for (int r = 0; r < R; ++r) {
            int m;
            if (std::scanf("%d %d", &lens[r], &m) != 2) return 1;
            start[r + 1] = start[r] + m;
        }
        std::vector<long long> begin(R + 1, 0);
        WindowParams p = {};
        p.lens = lens.data();
        p.query_start = start.data();
        p.begin = begin.data();
        p.R = R;
        p.Hkv = Hkv;
        p.G = G;
        p.Hq = Hkv * G;
        p.tokens = kRows / G;
        p.mbps = (1 << 27) - 128;
        p.max_q = max_q;
        p.T = start[R];
        p.grid = grid;
        long long total = 0;
        for (int r = 0; r < R; ++r) {
            begin[r] = total;
            total += request_cost<kLse>(p, r);
        }
        const long long share = begin[R] = even_share(total, grid, kLse);
        const size_t have = slots(Hkv, G, R, start[R]);
        std::vector<char> written(have, 0);
        long long wrote = 0, twice = 0, top = -1, stray = 0;
        for (int r = 0; r < R; ++r) {
            const Request x = request_of(p, r);
            for (int rb = 0; rb < row_blocks(p, x); ++rb)
                for (int h = 0; h < Hkv; ++h) {
                    const Cost c = lse_cost(p, x, rb, h, begin[r]);
                    for (long long b = c.at / share; b * share < c.end; ++b) {
                        const long long from = b * share > c.at ? b * share : c.at;
                        long long to = (b + 1) * share < c.end ? (b + 1) * share : c.end;
                        if (c.reaches(from) >= c.reaches(to)) continue;
                        const long long slot = lse_unit(p, x, rb, h) + b;
                        if (b >= grid || slot < 0 || (size_t)slot >= have) return 2;
                        twice += written[slot];
                        written[slot] = 1;
                        ++wrote;
                    }
                }
        }
        for (int r = 0; r < R; ++r) {
            const Request x = request_of(p, r);
            if (x.m < 0) continue;
            // resident rows: one item per head whether or not there are rows
            const int blocks = resident ? 1 : row_blocks(p, x);
            for (int rb = 0; rb < blocks; ++rb)
                for (int h = 0; h < Hkv; ++h) {
                    const RowParts v = row_parts(p, x, r, rb, h, share);
                    const long long first = (v.at - p.part) / kRows;
                    for (long long s = first; s < first + v.n; ++s) {
                        if (s > top) top = s;
                        if (s < 0 || (size_t)s >= have || !written[s]) ++stray;
                    }
                }
        }
        std::printf("%zu %lld %lld %lld %lld\n", have, wrote, twice, top, stray);
    }
    return 0;
}
