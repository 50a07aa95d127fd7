// The work items of the prefill kernels, from the lengths on the device: each
// request's new tokens, its row tiles and the table columns that a tile reads.
// Every function also compiles for the host, where a test holds the items of
// arbitrary words (lengths and starts are device data, which nobody has checked)
// against the bounds of the tables and of q.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mi {

struct PrefillBatch {
    const int32_t* context_lens;   // [R], counting the new tokens
    const int32_t* query_start;    // [R + 1]
    int G, mbps, T, max_q;
};

__host__ __device__ __forceinline__ int batch_word(const int32_t* at) {
#ifdef __CUDA_ARCH__
    return __ldg(at);
#else
    return *at;
#endif
}

// Request r's new tokens: rows q0 .. q0 + m - 1 of q; m < 0 where query_start is
// refused. (Bounds come before the difference, which any two words may wrap.)
struct NewTokens {
    int q0, m;
};
__host__ __device__ __forceinline__ NewTokens new_tokens(const PrefillBatch& p, int r) {
    const int q0 = batch_word(p.query_start + r), q1 = batch_word(p.query_start + r + 1);
    const bool ok = q0 >= 0 && q0 <= q1 && q1 <= p.T && q1 - q0 <= p.max_q;
    return {q0, ok ? q1 - q0 : -1};
}

// Its tokens, as many as a table row holds; none where the length is negative, so
// that positions of new tokens stay above -T.
__host__ __device__ __forceinline__ int held_tokens(const PrefillBatch& p, int r) {
    return min(max(batch_word(p.context_lens + r), 0), p.mbps * kBlock);
}

__host__ __device__ __forceinline__ int row_tiles(int rows, int tile_rows) {
    return rows > 0 ? (rows - 1) / tile_rows + 1 : 0;
}

// Row tile k (counted from the request's end) of request r: rows rho0 .. rho0 +
// rows_here - 1 of its nrows (token, head) rows; blocks 0 .. nblk - 1 of its table.
// False: past the first row, or nothing (m <= 0).
struct Item {
    int r, h, q0, m, n, first, nrows, rho0, rows_here, p_hi, nblk;
};
__host__ __device__ __forceinline__ bool tile_item(const PrefillBatch& p, int tile_rows, int r, int k, Item& it) {
    const NewTokens t = new_tokens(p, r);
    it.r = r;
    it.q0 = t.q0;
    it.m = t.m;
    it.nrows = max(t.m, 0) * p.G;
    const int tiles = row_tiles(it.nrows, tile_rows);
    if (k >= tiles) return false;
    it.n = held_tokens(p, r);
    it.first = it.n - it.m;  // position of new token 0 (negative only when m > n)
    it.rho0 = (tiles - 1 - k) * tile_rows;
    it.rows_here = min(tile_rows, it.nrows - it.rho0);
    it.p_hi = it.first + (it.rho0 + it.rows_here - 1) / p.G;  // position of the tile's last row
    it.nblk = it.p_hi >= 0 ? it.p_hi / kBlock + 1 : 0;        // blocks any row of the tile reads
    return true;
}

// Sliding windows: `rows` rows of a request and KV head; r < 0: no more.
struct SlideItem {
    int r, h, q0, first, n, p_hi;  // as Item
    int tok0, m;                   // the item's first of the request's m new tokens
    int head, gap, nblk;  // the blocks 0 .. head - 1 and from head + gap on, nblk in all
    int lo, sinks;        // tokens that some row of the request sees: below sinks, and from lo on
};

// A request's items per KV head; 0 where it is refused.
__host__ __device__ __forceinline__ int slide_tiles(const PrefillBatch& p, int r, int rows) {
    return row_tiles(max(new_tokens(p, r).m, 0) * p.G, rows);
}

// Item k, counted from the request's end, of its `tiles`, KV head h.
__host__ __device__ __forceinline__ SlideItem slide_tile_item(const PrefillBatch& p, int window, int sinks, int rows, int r,
                                                              int h, int tiles, int k) {
    SlideItem it;
    it.r = r;
    it.h = h;
    const NewTokens t = new_tokens(p, r);
    it.q0 = t.q0;
    it.m = t.m;
    it.n = held_tokens(p, r);
    it.first = it.n - it.m;
    it.tok0 = (tiles - 1 - k) * (rows / p.G);
    it.p_hi = it.first + min(it.tok0 + rows / p.G, it.m) - 1;
    auto window_of = [&](int pos) { return pos >= window ? pos - window + 1 : 0; };
    const int from = window_of(max(0, it.first + it.tok0));  // the first row's window
    it.head = (min(sinks, from) + kBlock - 1) / kBlock;
    const int all = it.p_hi >= 0 ? it.p_hi / kBlock + 1 : 0;
    it.gap = max(0, min(from / kBlock, all) - it.head);
    it.nblk = all - it.gap;
    it.lo = window_of(max(0, it.first));
    it.sinks = min(sinks, it.lo);
    return it;
}

}  // namespace mi
