// Cuts batches of a sliding decode on the host, with the kernel's own functions, and
// marks the places of all partial results. stdin: lines of "sms bytes Hkv G head_dim ulp B
// blocks[B]"; every quotient of the plan is off by up to `ulp` units in its last place. Prints
// per line: places of the workspace, pieces with partial results, the largest place, places
// marked twice, pieces found twice or not at all, whether the places were divisions, the
// first step and the other.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

#include "sliding_plan.cuh"

using namespace mi;

int main() {
    int sms, bytes, Hkv, G, hd, ulp, B;
    std::mt19937 rng(5);
    while (std::scanf("%d %d %d %d %d %d %d", &sms, &bytes, &Hkv, &G, &hd, &ulp, &B) == 7) {
        std::vector<int> nb(B);
        long long blocks = 0, units = 0;
        int largest = 0, smallest = 0x7FFFFFFF;
        for (int& x : nb) {
            if (std::scanf("%d", &x) != 1) return 1;
            blocks += (long long)Hkv * x;
            units += x > 0 ? Hkv : 0;
            largest = std::max(largest, x);
            smallest = std::min(smallest, x);
        }
        if (largest == 0) return 2;
        const int grid = kSlideBlocks * sms, warps = grid * kSlideWarps, most = slide_slots(sms);
        const CutSizes sizes = {(float)warps, (float)blocks, (float)units, largest, G * hd, slide_flow(hd, bytes), slide_alone(bytes)};
        auto quotient = [&](float a, float b) {
            float q = a / b;
            const int off = (int)(rng() % (2 * ulp + 1)) - ulp;
            for (int i = 0; i < std::abs(off); ++i) q = std::nextafterf(q, off < 0 ? 0.f : INFINITY);
            return q;
        };
        CutTry best = {INFINITY, 0.f, 0.f, 1.f};
        for (int lane = 0; lane < 32; ++lane) {
            const CutTry c = try_cut(sizes, lane, quotient);
            if (c.cost < best.cost) best = c;
        }
        const Cut cut(best, B, largest);
        const EvenCut even(cut, B, Hkv, smallest, largest);
        std::vector<char> place(most, 0);
        long long split = 0, top = -1, twice = 0, lost = 0;
        auto mark = [&](long long at) {
            ++split;
            top = std::max(top, at);
            if (at < 0) return;
            if (at < most) twice += place[at]++ > 0;
        };
        long long first_split = 0;
        std::vector<long long> first(B + 1, 0), slot(B, 0);
        for (int b = 0; b < B; ++b) {
            const int np = cut.pieces(b, nb[b]);
            slot[b] = first_split;
            if (np < (nb[b] > 0)) return 3;
            first[b + 1] = first[b] + (long long)Hkv * np;
            if (np > 1) first_split += (long long)Hkv * np;
        }
        if (even.even) {
            lost += even.total(B) != first[B] || even.split(B) != first_split;
            std::vector<char> seen(first[B], 0);
            for (int x = 0; x < even.total(B); ++x) {
                int b, o, at;
                even.find(x, b, o, at);
                if (b < 0 || b >= B || first[b] + o != x) {
                    ++lost;
                    continue;
                }
                lost += seen[x]++ > 0;
                const int np = cut.pieces(b, nb[b]), h = o / np;
                if (np > 1) mark(at + (long long)h * np + (o - h * np));
            }
        } else {
            for (int b = 0; b < B; ++b) {
                const int np = cut.pieces(b, nb[b]);
                for (int o = 0; np > 1 && o < Hkv * np; ++o) mark(slot[b] + o);
            }
        }
        std::printf("%d %lld %lld %lld %lld %d %d %d\n", most, split, top, twice, lost, (int)even.even, cut.step, cut.tail_step);
    }
    return 0;
}
