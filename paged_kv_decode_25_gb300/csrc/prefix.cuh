// The work items of attention over shared prefixes, (group, tile of requests,
// split of the prefix, KV head), found by every block itself from the groups
// and lengths on the device.
#pragma once

#include "batch.cuh"

namespace mi {

constexpr int kSplitStep = 8;  // blocks: a split is whole 128-key stages

struct PrefixWork {
    const int32_t* lens = nullptr;    // [P] tokens of each prefix
    const int32_t* starts = nullptr;  // [P + 1] the groups' requests
    int4* rows = nullptr;             // [B] see DecodeExt
    float* part = nullptr;            // [slots][slot_rows][HD]
    float* part_lse = nullptr;        // [slots][slot_rows]
    int P = 0, B = 0, sms = 0;
};

// Item: prefix g's keys from its block blk0 on (n tokens there), against the
// `count` requests from b0 on, KV head h; results go to slot `slot`.
struct PrefixItem {
    int g, h, b0, count, blk0, n, slot;
};

// Slots for B requests in P groups, `per` requests a tile: the items of
// prefix_plan, whose splits are at least total / (2 sms) blocks long, are at
// most 2 sms and one more for every (tile, head).
inline long long prefix_slots(int B, int Hkv, int P, int per, int sms) {
    return 2LL * sms + (long long)Hkv * ((B + per - 1) / per + P);
}

__device__ __forceinline__ int prefix_tokens(const PrefixWork& w, int mbps, int g) {
    return min(max(__ldg(w.lens + g), 0), mbps * kBlock);
}
// Items of group g for splits of `step` blocks.
__device__ __forceinline__ long long prefix_items(const PrefixWork& w, int Hkv, int mbps, int per, long long step, int g) {
    const int tiles = (__ldg(w.starts + g + 1) - __ldg(w.starts + g) + per - 1) / per;
    return (long long)Hkv * tiles * (((prefix_tokens(w, mbps, g) + kBlock - 1) / kBlock + step - 1) / step);
}

// Plans the call in every block, with all its threads: the blocks of a split
// in `step`, the items laid end to end in `sums`, their number returned.
// Writes the requests' rows.
__device__ inline long long prefix_plan(const PrefixWork& w, int Hkv, int G, int mbps, int per, int32_t* dev_err,
                                        long long* sums, long long& step) {
    const int tid = threadIdx.x, nt = blockDim.x;
    const int gtid = blockIdx.x * nt + tid, nthreads = gridDim.x * nt;
    if (!starts_ascend(w.starts, w.P, w.B)) {
        // no request's prefix is known
        if (gtid == 0) raise_err(dev_err, MI_DEVERR_BAD_QUERY);
        for (int b = gtid; b < w.B; b += nthreads) w.rows[b] = make_int4(0, 0, 0, 0);
        return 0;
    }
    // The split length: short enough that the grid has work, long enough that
    // one wave takes it all. Start from an even share; a share that leaves
    // more items than SMs (each group rounds up) grows by that ratio.
    auto rounded = [](long long x) { return max((x + kSplitStep - 1) / kSplitStep, 1ll) * kSplitStep; };
    auto items = [&](int g) { return prefix_items(w, Hkv, mbps, per, step, g); };
    step = 1;
    const long long cost = flat_scan(w.P, items, sums);  // blocks times tiles and heads
    __syncthreads();
    step = 1ll << 40;
    const long long units = flat_scan(w.P, items, sums);
    const long long target = units < w.sms ? w.sms : 2LL * w.sms;
    step = rounded((cost + target - 1) / target);
    __syncthreads();
    long long total = flat_scan(w.P, items, sums);
    for (int round = 0; round < 3 && units < w.sms && total > w.sms; ++round) {
        step = rounded((step * total + w.sms - 1) / w.sms);
        __syncthreads();
        total = flat_scan(w.P, items, sums);
    }
    for (int g = gtid; g < w.P; g += nthreads)
        if (__ldg(w.lens + g) > mbps * kBlock) raise_err(dev_err, MI_DEVERR_BAD_CONTEXT);
    // each request's slots; those outside every group have none
    const int b_first = __ldg(w.starts), b_last = __ldg(w.starts + w.P);
    for (int b = gtid; b < w.B; b += nthreads) {
        int4 at = make_int4(0, 0, 0, 0);
        if (b >= b_first && b < b_last) {
            int lo = 0, hi = w.P;  // starts[lo] <= b < starts[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(w.starts + mid) <= b) lo = mid;
                else hi = mid;
            }
            const int splits = (int)(((prefix_tokens(w, mbps, lo) + kBlock - 1) / kBlock + step - 1) / step);
            if (splits > 0) {
                const long long first = flat_before(w.P, items, sums, lo);
                const int i = b - __ldg(w.starts + lo);
                at = make_int4((int)first + (i / per) * splits * Hkv, splits, (i % per) * G, 0);
            }
        }
        w.rows[b] = at;
    }
    return total;
}

// Item x of the plan.
__device__ inline PrefixItem prefix_item(const PrefixWork& w, int Hkv, int mbps, int per, const long long* sums,
                                         long long step, long long x) {
    PrefixItem it;
    long long first;
    it.g = flat_find(w.P, [&](int g) { return prefix_items(w, Hkv, mbps, per, step, g); }, sums, x, first);
    it.slot = (int)x;
    const int n = prefix_tokens(w, mbps, it.g), o = (int)(x - first);
    const int splits = (int)(((n + kBlock - 1) / kBlock + step - 1) / step);
    const int s = o / Hkv % splits, tile = o / Hkv / splits;
    it.h = o % Hkv;
    it.b0 = __ldg(w.starts + it.g) + tile * per;
    it.count = min(__ldg(w.starts + it.g + 1) - it.b0, per);
    it.blk0 = (int)(s * step);
    it.n = (int)min((long long)n - (long long)it.blk0 * kBlock, step * kBlock);
    return it;
}

// The prefix part of a shared-prefix decode step: each slot's partial outputs
// and log-sum-exps (prefill.cu). `slots` as prefix_slots for tiles of
// prefix_tile_requests(G) requests.
constexpr int prefix_tile_requests(int G) { return 2 * (128 / G); }
mi_status prefix_partials(const mi_dims* dims, int32_t max_prefix_blocks, const void* q, const void* k_cache,
                          const void* v_cache, const int32_t* prefix_tables, float scale, const PrefixWork& work,
                          long long slots, int32_t* dev_err, mi_stream_t stream);

}  // namespace mi
