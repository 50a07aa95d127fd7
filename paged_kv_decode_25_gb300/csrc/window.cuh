// The plan of mi_paged_prefill_scores' first launch and of those that read its
// results: each request's rows and keys, their cost, and the slots of partial
// log-sum-exps. Every function also compiles for the host, where a test walks
// the plan of whole batches and holds every slot that is read against those that
// were written.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mi {
namespace window {

constexpr int kLse = 0, kSum = 1, kWindow = 2;
constexpr int kKeys = 128;        // keys of a tile
constexpr int kRows = 256;        // rows of a block of query rows: whole tokens, kRows / G of them
constexpr int kMostBlocks = 256;  // of the grid, whatever the device has

__host__ __device__ __forceinline__ int load(const int32_t* at) {
#ifdef __CUDA_ARCH__
    return __ldg(at);
#else
    return *at;
#endif
}
// (written by the launch before)
__host__ __device__ __forceinline__ long long load_cg(const long long* at) {
#ifdef __CUDA_ARCH__
    return __ldcg(at);
#else
    return *at;
#endif
}

// Slots of partial log-sum-exps, kRows each, of a call: its units and blocks.
inline size_t slots(int Hkv, int G, int R, int total_q) {
    return (size_t)Hkv * ((size_t)total_q / (kRows / G) + R) + kMostBlocks;
}

struct WindowParams {
    const int32_t* tables;         // [R][mbps]
    const int32_t* lens;           // [R]
    const int32_t* query_start;    // [R + 1]
    float* part;                   // [slots][kRows] partial log-sum-exps, base 2 (see Cost)
    float* nlse;                   // [Hkv][T][G] the rows' negated log-sum-exps (-inf: no key)
    unsigned int* next;            // kSum: the next item
    long long* begin;              // [R + 1] the cost before each request, then a block's share (0: bad query_start)
    float* scores;                 // [num_blocks][Hkv][16]
    int32_t* dev_err;
    int R, Hq, Hkv, G, num_blocks, mbps, T, max_q, fresh;
    int tokens;                    // of a row block: kRows / G
    int xt;                        // kWindow: 128-row halves that hold rows
    int grid;
    float sl2;                     // scale * log2(e), never 0
    long long wait_ns;
    int withhold;                  // failure-detection test: the first Y tile of every block is not announced
};

// Request r: n tokens, the last m of them with queries in rows q0 .. q0+m-1;
// first = n - m (negative: the rows before position 0 see nothing). A request
// with more queries than the call allows has m = -1 and is left alone.
// (Divisions by the tokens of a row block are made once: the plans ran for 3 and
// 5 us with them where they are used.)
struct Request {
    int n, m, q0, first;
    int full, rest;  // whole row blocks, tokens of the last one besides
    int before;      // bounds the row blocks of the requests before this one
};

__host__ __device__ __forceinline__ Request request_of(const WindowParams& p, int r) {
    Request x;
    x.q0 = load(p.query_start + r);
    x.m = load(p.query_start + r + 1) - x.q0;
    x.n = min(max(load(p.lens + r), 0), p.mbps * kBlock);
    x.first = x.n - x.m;
    if (x.m < 0 || x.m > p.max_q) x.m = -1;
    x.full = max(x.m, 0) / p.tokens;
    x.rest = max(x.m, 0) - x.full * p.tokens;
    x.before = x.q0 / p.tokens + r;
    return x;
}

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Blocks of query rows.
__host__ __device__ __forceinline__ int row_blocks(const WindowParams& p, const Request& x) {
    return x.full + (x.rest > 0);
}
// 256-key stages that the rows of block rb see.
__host__ __device__ __forceinline__ int seen_stages(const WindowParams& p, const Request& x, int rb) {
    const int last = x.first + min(x.m, (rb + 1) * p.tokens) - 1;
    return last >= 0 ? last / (2 * kKeys) + 1 : 0;
}

// The shares of kLse and kWindow. Their work lies end to end as units (request,
// row block, head), each costing its products and its own start; block b of the
// grid takes the cost from b to b + 1 shares, wherever that begins and ends
// within a unit. So all blocks end together (whole splits of equal length, dealt
// out, left some with a quarter more than the mean), and a row's keys are split
// only where a share ends. Units and blocks both ascend along the work, so
// u + b numbers the pairs that meet: the slots of partial log-sum-exps.
//
// The cost of kLse is in keys times row tiles, closed in form over a request's
// row blocks: a prompt has thousands. (Stages round it up; a share may be off by
// one.)
constexpr int kUnitCost = 1050;   // X's copy, the pipeline's start, the first maximum, the last tiles' masks: 7,000
                                  // clocks, where a tile of 256 keys takes 1,700
constexpr int kUnitTiles = 2;     // kWindow: X's copy and the pipeline's start, in stages
constexpr int kLeastCost = 1024, kLeastTiles = 6;  // of a share
static_assert(kLeastCost > 4 * kKeys, "a share has part of a stage's end wherever it begins");

// Row tiles of a request's last row block.
__host__ __device__ __forceinline__ int last_tiles(const WindowParams& p, const Request& x) {
    return x.rest > 0 && x.rest * p.G <= kKeys ? 1 : 2;
}
// Cost of one head's first k row blocks.
__host__ __device__ __forceinline__ long long cost_before(const WindowParams& p, const Request& x, int k) {
    const long long t = p.tokens, f = max(x.first, 0), full = min(k, x.full);
    long long v = full * (kUnitCost + 2 * f) + t * full * (full + 1);
    if (k > full) v += kUnitCost + last_tiles(p, x) * (f + x.m);
    return v;
}
// a / d, at most a few hundred
__host__ __device__ __forceinline__ int small_quotient(long long a, long long d) {
    int q = (int)((float)a / (float)d);
    while ((q + 1) * d <= a) ++q;
    while (q * d > a) --q;
    return q;
}
// A unit: its cost from `at` on, `keys` cost units to a stage after `start`.
struct Cost {
    long long at, end;
    int start, per, stages;
    // the stage that the work up to c reaches
    __host__ __device__ int reaches(long long c) const {
        const long long q = c - at - start;
        return q <= 0 ? 0 : (int)min((long long)stages, (q + per - 1) / per);
    }
};
__host__ __device__ __forceinline__ Cost lse_cost(const WindowParams& p, const Request& x, int rb, int h, long long begin) {
    Cost c;
    const long long before = cost_before(p, x, rb), w = cost_before(p, x, rb + 1) - before;
    c.at = begin + p.Hkv * before + h * w;
    c.end = c.at + w;
    c.start = kUnitCost;
    c.per = 2 * kKeys * (rb == x.full ? last_tiles(p, x) : 2);
    c.stages = seen_stages(p, x, rb);
    return c;
}
__host__ __device__ __forceinline__ int lse_unit(const WindowParams& p, const Request& x, int rb, int h) {
    return h + p.Hkv * (rb + x.before);
}
template <int MODE>
__host__ __device__ __forceinline__ long long request_cost(const WindowParams& p, int r) {
    const Request x = request_of(p, r);
    if (MODE == kLse) return x.m > 0 ? p.Hkv * cost_before(p, x, row_blocks(p, x)) : 0;
    return x.m < 0 ? 0 : (long long)p.Hkv * (kUnitTiles + ceil_div(x.n, kKeys));
}
// A block's share of the cost (a little above total / grid, as fp32 may round it down).
__host__ __device__ __forceinline__ long long even_share(long long total, int grid, int mode) {
    return max((long long)((float)total / (float)grid * 1.000001f) + 1, (long long)(mode == kLse ? kLeastCost : kLeastTiles));
}

// The partial log-sum-exps of a row block, from the blocks that had keys of it:
// those of its first and last stage, and all between (a share is longer than a
// stage). A request without query tokens has no row block, so no unit and no
// cost: nothing was written for it, and its place in the cost means nothing.
struct RowParts {
    const float* at;
    int n;
};
__host__ __device__ __forceinline__ RowParts row_parts(const WindowParams& p, const Request& x, int r, int rb, int h,
                                                       long long share) {
    if (rb >= row_blocks(p, x)) return RowParts{p.part, 0};
    const Cost c = lse_cost(p, x, rb, h, load_cg(p.begin + r));
    const int b0 = small_quotient(c.at + c.start, share);
    RowParts v;
    v.n = c.stages > 0 ? small_quotient(c.at + c.start + (c.stages - 1LL) * c.per, share) - b0 + 1 : 0;
    v.at = p.part + (long long)(lse_unit(p, x, rb, h) + b0) * kRows;
    return v;
}

}  // namespace window
}  // namespace mi
