// How a sliding decode cuts its units, (request, KV head)s, into pieces, and where
// the pieces' partial results go. Every function also compiles for the host, where
// a test cuts whole batches and holds every place against the workspace's.
#pragma once

#include <cuda_runtime.h>

namespace mi {

constexpr int kSlideWarps = 4;
// Blocks per SM. (Four for one-byte caches, at 128 registers a thread: 116 us on the
// device instead of 92 for 128 windows of 4,096 tokens, 4 KV heads, e4m3.)
constexpr int kSlideBlocks = 3;
// Pieces that have partial results, at most, per warp of the grid.
constexpr int kSplitPerWarp = 8;

// Partial results that the workspace has room for.
__host__ __device__ constexpr int slide_slots(int sms) { return kSplitPerWarp * kSlideWarps * kSlideBlocks * sms + 64; }

// In a warp's block times: a piece's own cost (its queries, its output), that of a
// split unit's end, and of adding up 512 outputs of a piece there. Fitted, with
// CutSizes::alone, to 15 shapes (1 to 256 requests, windows of 128 to 4,096, the three
// types) cut into 1 to 24 pieces: the plan's choice is within 0.9 % of the best one on
// average. (More rounds of shorter pieces lose to one round: each costs its results and
// counts, and the additions fall to the blocks that end last.)
constexpr float kPieceCost = 16.f, kSplitCost = 1.f, kMergeCost = 0.1f;

// A block's time at full memory rate over its time in a warp, for heads of hd elements
// of `bytes`: 6.8 TB/s; a warp's block takes about 0.75 us (bf16: its ring's latency,
// whoever else is there) or 1 (one-byte codes, of which an SM's warps share the time: 128
// windows of 4,096 in e4m3 take 0.65 us a block with 3.4 warps an SM, 0.88 with 6.7, 1.05
// with 10.1, 1.3 with 12).
inline float slide_flow(int hd, int bytes) {
    return (float)(2 * 16 * hd * bytes) / 6.8e12f / (bytes == 2 ? 0.75e-6f : 1e-6f);
}
// A warp's share of a block's time which others on its SM do not lengthen.
inline float slide_alone(int bytes) { return bytes == 2 ? 1.f : 0.6f; }

// What the choice depends on.
struct CutSizes {
    float warps, blocks, units;  // of the grid; in sight of all units; with any
    int largest;                 // blocks in sight of a unit
    int outs;                    // G * head_dim
    float flow, alone;           // slide_flow, slide_alone
};

// A way to cut: blocks of a piece, for the first `part` of the requests and for the others.
struct CutTry {
    float cost, step, tail_step, part;
};

// Lane 0 to 31 tries 1 to 16 pieces for the largest unit, or 16 to 448 in steps of a
// quarter. Warps take whole pieces in turn; what the last round leaves over is cut so
// that every warp has some of it. The time is that of the rounds, or of all bytes at
// the memory's rate, and the end of the unit with the most pieces.
// No cut is finer than `least`: a split unit of nb > step blocks has fewer than 2 nb /
// step pieces, so all of them together stay within kSplitPerWarp a warp, and roundings
// of `least` within the 64 places besides. div: a quotient, to two ulp.
template <class Div>
__host__ __device__ __forceinline__ CutTry try_cut(const CutSizes& z, int lane, Div div) {
    const float all = z.blocks * z.flow;  // time of all blocks at the memory's rate, in a warp's block times
    const float np = lane < 16 ? (float)(lane + 1) : (float)((16 + 4 * (lane & 3)) << ((lane - 16) >> 2));
    const float big = (float)z.largest;
    const float least = fmaxf(1.f, ceilf(div(2.f * z.blocks, (float)kSplitPerWarp * z.warps)));
    const float step = fmaxf(least, ceilf(div(big, np)));
    const float most = ceilf(div(big, step)), outs = (float)((z.outs + 511) / 512);
    auto end_cost = [&](float pieces) { return pieces > 1.f ? kSplitCost + kMergeCost * pieces * outs : 0.f; };
    // the largest units have `most` pieces, the others half a piece more than their share
    const float fill = div(z.blocks, z.units * big);
    const float rounds = div(fmaxf(z.units * (most * fill + 0.5f * (1.f - fill)), z.units), z.warps);
    const float whole = floorf(rounds), over = rounds - whole;
    CutTry c = {0.f, step, step, 1.f};
    const float last = over > 0.f ? z.alone + (1.f - z.alone) * over : 0.f;
    c.cost = fmaxf(all, (whole + last) * (step + kPieceCost)) + end_cost(most);
    if (whole > 0.f && over > 0.01f) {
        const float tail_np = fminf(16.f, div(most * fill, over));  // so that they fill a round
        const float s = fminf(step, fmaxf(least, ceilf(div(big, fmaxf(1.f, tail_np)))));
        const float cost = fmaxf(all, whole * (step + kPieceCost) + s + kPieceCost) +
                           end_cost(fmaxf(most, ceilf(div(big, s))));
        if (cost < c.cost) {
            c.cost = cost;
            c.tail_step = s;
            c.part = div(whole, rounds);
        }
    }
    c.cost += 0.01f * most;
    return c;
}

// The blocks of a piece, for requests before b0 and for those from it on. (A step of
// the largest unit or more is no cut. With very many heads of long tables it may be
// past what an int holds.)
struct Cut {
    int step, tail_step, b0;
    __host__ __device__ Cut(const CutTry& c, int B, int largest)
        : step(blocks(c.step, largest)), tail_step(blocks(c.tail_step, largest)),
          b0(c.part < 1.f ? min(B, (int)(c.part * (float)B)) : B) {}
    __host__ __device__ static int blocks(float step, int largest) {
        return step < (float)largest ? max(1, (int)step) : largest;
    }
    __host__ __device__ int pieces(int b, int nb) const {
        const int s = b < b0 ? step : tail_step;
        return (nb + s - 1) / s;
    }
};

// As a rule every context is longer than the window, and every request before b0 has
// as many pieces as any other, and so from it on: then places are divisions.
struct EvenCut {
    int b0, n0, n1;        // pieces of a unit before request b0, and from it on
    int per0, per1, head;  // of a request; of all before b0
    bool even;
    __host__ __device__ EvenCut(const Cut& cut, int B, int Hkv, int smallest, int largest)
        : b0(cut.b0), n0(cut.pieces(0, largest)), n1(cut.pieces(B, largest)), per0(Hkv * n0), per1(Hkv * n1), head(b0 * per0),
          even(cut.pieces(0, smallest) == n0 && cut.pieces(B, smallest) == n1 && smallest > 0) {}
    __host__ __device__ int total(int B) const { return head + (B - b0) * per1; }
    // pieces that have partial results
    __host__ __device__ long long split(int B) const {
        return (n0 > 1 ? (long long)b0 * per0 : 0) + (n1 > 1 ? (long long)(B - b0) * per1 : 0);
    }
    // Piece x: its request, its number among the request's, and the place of the
    // request's first partial result (meaningless without a split).
    __host__ __device__ void find(int x, int& b, int& o, int& slot) const {
        const bool tail = x >= head;
        const int y = tail ? x - head : x, per = tail ? per1 : per0, r = y / per;
        b = tail ? b0 + r : r;
        o = y - r * per;
        slot = x - o - (tail && n0 == 1 ? head : 0);
    }
};

}  // namespace mi
