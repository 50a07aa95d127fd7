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
    // [B] {first slot, splits, row in the slot, 0}: split s of KV head h is slot
    // first + s * Hkv + h
    int4* rows = nullptr;
    float* part = nullptr;            // [slots][slot_rows][HD], normalised
    float* part_lse = nullptr;        // [slots][slot_rows] log2-sum-exps
    const int32_t* own = nullptr;     // [B] the requests' own tokens (at most own_blocks blocks each)
    int P = 0, B = 0, sms = 0, own_blocks = 0;
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
__device__ __forceinline__ int prefix_blocks(const PrefixWork& w, int mbps, int g) {
    return (prefix_tokens(w, mbps, g) + kBlock - 1) / kBlock;
}
// Tiles of group g's requests, all KV heads counted. (The last group may end
// before it starts: it is empty.)
__device__ __forceinline__ int prefix_units(const PrefixWork& w, int Hkv, int per, int g) {
    return Hkv * ((max(__ldg(w.starts + g + 1) - __ldg(w.starts + g), 0) + per - 1) / per);
}
// The first request behind all groups.
__device__ __forceinline__ int prefix_end(const PrefixWork& w) {
    return max(__ldg(w.starts + w.P), __ldg(w.starts + max(w.P - 1, 0)));
}
__device__ __forceinline__ int prefix_splits(int blocks, int step) { return (blocks + step - 1) / step; }
// Items of group g for splits of `step` blocks.
__device__ __forceinline__ long long prefix_items(const PrefixWork& w, int Hkv, int mbps, int per, int step, int g) {
    return (long long)prefix_units(w, Hkv, per, g) * prefix_splits(prefix_blocks(w, mbps, g), step);
}

// Item x of the plan, whose items lie end to end in `sums`.
__device__ inline PrefixItem prefix_item(const PrefixWork& w, int Hkv, int mbps, int per, const long long* sums,
                                         int step, long long x) {
    PrefixItem it;
    long long first;
    it.g = flat_find(w.P, [&](int g) { return prefix_items(w, Hkv, mbps, per, step, g); }, sums, x, first);
    it.slot = (int)x;
    const int n = prefix_tokens(w, mbps, it.g), o = (int)(x - first), splits = prefix_splits((n + kBlock - 1) / kBlock, step);
    const int st = o / Hkv, tile = st / splits;
    it.h = o - st * Hkv;
    it.b0 = __ldg(w.starts + it.g) + tile * per;
    it.count = min(__ldg(w.starts + it.g + 1) - it.b0, per);
    it.blk0 = (st - tile * splits) * step;
    it.n = (int)min((long long)n - (long long)it.blk0 * kBlock, (long long)step * kBlock);
    return it;
}

// Blocks of a split, of whole stages, no shorter than `share`.
__device__ __forceinline__ int prefix_step(float share) {
    // (a table has at most 2^27 blocks)
    return (int)fminf(fmaxf(ceilf(share * (1.f / kSplitStep)), 1.f), (float)((1 << 27) / kSplitStep)) * kSplitStep;
}

// The SMs that the prefix part takes. The requests' own tokens are read by a
// launch that fills the SMs this one leaves (decode.cu). The two are bound by
// different things, tensor cores and memory, and share the SMs in proportion
// to their work, so that both end together: a (tile, block) of the prefix takes
// an SM as long as kTileBlock blocks of own tokens. Own tokens get 11 of 15 SMs
// at most: where they are most of the work they are bound by memory, and the
// prefix part's start alone is 12 us. Measured on the device with 64 chats of 32
// to 1,024 tokens behind 4,100, 128 of 16 to 512 behind 32,000, and 90 in six
// groups: 34, 83 and 33 us (one part after the other 44, 96 and 41); kTileBlock
// 1: 35-38, 87, 34; 2: 34, 90, 33; with 3 of 4 SMs the chats take 37, with 2 of
// 3 40. (On 152 SMs 11 of 15 leave the prefix part 41, room for eight KV heads
// with one tile in five splits, 40 items; 3 of 4 leave 38 and four splits. The
// cap fits such counts and is neutral for 2, 4 and 16 units, by the plan's own
// cost: a number found by trying, not a rule.)
constexpr float kTileBlock = 1.8f;
__device__ __forceinline__ int prefix_budget(const PrefixWork& w, float tile_blocks, float own_blocks) {
    const float a = tile_blocks * kTileBlock, b = own_blocks;
    if (a + b <= 0.f) return w.sms;
    const int least = max(w.sms - w.sms * 11 / 15, 1), x = (int)((float)w.sms * (a / (a + b)) + 0.5f);
    return min(max(x, least), w.sms);
}
__device__ __forceinline__ int own_blocks_of(const PrefixWork& w, int b) {
    return (min(max(__ldg(w.own + b), 0), w.own_blocks * kBlock) + kBlock - 1) / kBlock;
}

// An item's prologue and end count as much as this many blocks of its prefix
// (6 us, and 1.7 us for 8 blocks).
constexpr int kItemBlocks = 27;

// Plans the call in every block, with all its threads: the blocks of a split
// in `step`, the grid's blocks that take items (the first ones) in `active`,
// the items laid end to end in `sums` (two words more than flat_words), their
// number returned, this block's first one in *mine (shared). Writes the
// requests' rows. Up to 32 groups one warp does it from one load of each group's
// numbers: the block's other way, four scans of the list, took 3 us of a call.
__device__ inline long long prefix_plan(const PrefixWork& w, int Hkv, int G, int mbps, int per, int32_t* dev_err,
                                        long long* sums, int& step, int& active, PrefixItem* mine) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
    auto no_prefix = [&]() {  // no request's prefix is known
        if (blockIdx.x == 0 && tid == 0) raise_err(dev_err, MI_DEVERR_BAD_QUERY);
        for (int b = blockIdx.x * nt + tid; b < w.B; b += gridDim.x * nt) w.rows[b] = make_int4(0, 0, 0, 0);
    };
    long long total = 0;
    if (w.P <= 32) {
        if (tid < 32) {
            const bool in = lane < w.P;
            const int s0 = __ldg(w.starts + min(lane, w.P)), len = in ? __ldg(w.lens + lane) : 0;
            int s1 = __shfl_down_sync(0xffffffffu, s0, 1);
            if (lane == 31) s1 = __ldg(w.starts + w.P);  // (read by lane 31 alone when there are 32 groups)
            const bool bad = s0 < 0 || s0 > w.B || (in && (s1 < 0 || s1 > w.B || (s1 < s0 && lane < w.P - 1)));
            s1 = max(s1, s0);
            if (__any_sync(0xffffffffu, bad)) {
                step = 0;
            } else {
                const int units = in ? Hkv * ((s1 - s0 + per - 1) / per) : 0;
                const int blocks = (min(max(len, 0), mbps * kBlock) + kBlock - 1) / kBlock;
                if (blockIdx.x == 0 && in && len > mbps * kBlock) raise_err(dev_err, MI_DEVERR_BAD_CONTEXT);
                auto sum = [](float v) {
#pragma unroll 1
                    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    return v;
                };
                float own = 0.f;
                for (int b = lane; b < w.B; b += 32) own += (float)own_blocks_of(w, b);
                const float cost = sum((float)units * (float)blocks);
                active = prefix_budget(w, cost, sum(own) * (float)Hkv);
                step = kSplitStep;
                if ((int)blockIdx.x < active) {  // the others are done, and make room
                    // lane i tries a share of 0.5 + i / 20 of the even one, made
                    // as short as its number of splits of the longest prefix
                    // allows; never so short that the slots would not do (the
                    // factor is for the rounding of `cost`)
                    const int longest = max(__reduce_max_sync(0xffffffffu, blocks), 1);
                    const int least = prefix_step(cost * 1.00001f / (float)(2 * w.sms));
                    const int tried = prefix_step(cost / (float)active * (float)(10 + lane) * 0.05f);
                    step = max(least, prefix_step((float)((longest + prefix_splits(longest, tried) - 1) / prefix_splits(longest, tried))));
                    int items = 0;
                    for (int g = 0; g < w.P; ++g)
                        items += __shfl_sync(0xffffffffu, units, g) * prefix_splits(__shfl_sync(0xffffffffu, blocks, g), step);
                    // the least time, then the longest split
                    const float time = (float)((items + active - 1) / active) * (float)(min(step, longest) + kItemBlocks);
                    const unsigned best = __reduce_min_sync(0xffffffffu, __float_as_uint(time));
                    step = (int)__reduce_max_sync(0xffffffffu, __float_as_uint(time) == best ? (unsigned)step : 0u);
                    items = units * prefix_splits(blocks, step);
                    total = __reduce_add_sync(0xffffffffu, items);
                    int x = items;
#pragma unroll 1
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += y;
                    }
                    sums[lane] = x - items;
                    if (lane == 31) sums[32] = x;
                    __syncwarp();
                    if (lane == 0 && blockIdx.x < total) *mine = prefix_item(w, Hkv, mbps, per, sums, step, blockIdx.x);
                }
            }
            if (lane == 0) {
                sums[33] = step;
                sums[34] = total;
                sums[35] = active;
            }
        }
        __syncthreads();
        step = (int)sums[33];
        total = sums[34];
        active = (int)sums[35];
        if (step == 0) {
            no_prefix();
            return 0;
        }
    } else {
        const int end = __ldg(w.starts + w.P);
        if (!starts_ascend(w.starts, w.P - 1, w.B) || end < 0 || end > w.B) {
            no_prefix();
            return 0;
        }
        const long long cost = flat_scan(
            w.P, [&](int g) { return (long long)prefix_units(w, Hkv, per, g) * prefix_blocks(w, mbps, g); }, sums);
        __syncthreads();
        active = prefix_budget(
            w, (float)cost, (float)(Hkv * flat_scan(w.B, [&](int b) { return (long long)own_blocks_of(w, b); }, sums)));
        __syncthreads();
        auto items = [&](int g) { return prefix_items(w, Hkv, mbps, per, step, g); };
        // an even share
        step = prefix_step((float)cost * 1.00001f / (float)active);
        total = flat_scan(w.P, items, sums);
        for (int g = blockIdx.x * nt + tid; g < w.P; g += gridDim.x * nt)
            if (__ldg(w.lens + g) > mbps * kBlock) raise_err(dev_err, MI_DEVERR_BAD_CONTEXT);
        if (tid == 0 && blockIdx.x < min(total, (long long)active)) *mine = prefix_item(w, Hkv, mbps, per, sums, step, blockIdx.x);
        __syncthreads();
    }
    if ((int)blockIdx.x >= active) return 0;
    // each request's slots; those outside every group have none
    for (int b = blockIdx.x + active * tid; b < w.B; b += active * nt) {
        int4 at = make_int4(0, 0, 0, 0);
        if (b >= __ldg(w.starts) && b < prefix_end(w)) {
            int lo = 0, hi = w.P;  // starts[lo] <= b < starts[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(w.starts + mid) <= b) lo = mid;
                else hi = mid;
            }
            const int splits = prefix_splits(prefix_blocks(w, mbps, lo), step);
            if (splits > 0) {
                const long long first =
                    flat_before(w.P, [&](int g) { return prefix_items(w, Hkv, mbps, per, step, g); }, sums, lo);
                const int i = b - __ldg(w.starts + lo);
                at = make_int4((int)first + (i / per) * splits * Hkv, splits, (i % per) * G, 0);
            }
        }
        w.rows[b] = at;
    }
    return total;
}

// The prefix part of a shared-prefix decode step: each slot's partial outputs
// and log-sum-exps (prefill.cu). `slots` as prefix_slots for tiles of
// prefix_tile_requests(G) requests.
__host__ __device__ constexpr int prefix_tile_requests(int G) { return 2 * (128 / G); }
mi_status prefix_partials(const mi_dims* dims, int32_t max_prefix_blocks, const void* q, const void* k_cache,
                          const void* v_cache, const int32_t* prefix_tables, float scale, const PrefixWork& work,
                          long long slots, int32_t* dev_err, mi_stream_t stream);

}  // namespace mi
