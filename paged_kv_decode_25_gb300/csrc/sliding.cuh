// Which cached tokens a sliding window with sinks leaves in sight, in blocks: the
// one definition that the decode and prefill kernels and the host's sizes share.
#pragma once

#include "common.cuh"

namespace mi {

// What the token at position last sees: tokens 0 .. sinks - 1 and lo .. last. The
// blocks that hold any of them are 0 .. head - 1 and head + gap .. head + gap +
// blocks - head - 1 of its table; `gap` blocks in between are not looked at.
struct Sight {
    int sinks, lo, n;       // sinks <= lo: nothing is counted twice; n = last + 1
    int head, gap, blocks;  // blocks: how many hold something in sight
    __host__ __device__ Sight(int n_, int window, int sinks_) : n(n_) {
        lo = n > window ? n - window : 0;
        sinks = sinks_ < lo ? sinks_ : lo;
        const int all = n / kBlock + (n % kBlock != 0);
        head = sinks / kBlock + (sinks % kBlock != 0);
        gap = lo / kBlock > head ? lo / kBlock - head : 0;
        blocks = all - gap;
    }
    __device__ int column(int j) const { return j < head ? j : j + gap; }
    // Bit t: whether token 16 * column + t is in sight.
    __device__ uint32_t mask(int column) const {
        const int t0 = column * kBlock;
        return first_bits(n - t0) & (first_bits(sinks - t0) | ~first_bits(lo - t0));
    }
    static __device__ uint32_t first_bits(int k) { return k >= kBlock ? 0xFFFFu : (k <= 0 ? 0u : (1u << k) - 1u); }
};

}  // namespace mi
