// mi_paged_prefill_scores: the attention weight every cached token receives
// from many query tokens at once (the last tokens of a prompt, or all of it).
//
//   score[r][h][t] (+)= sum over query tokens i of request r with t <= pos_i
//                       and the G query heads j of h of 2^(x_ijt - lse_ij)
//
// A weight needs its row's log-sum-exp over all keys, so the logits x are
// computed twice: the first launch reduces them over the keys of each row, the
// last over the rows of each key (a small one between merges split rows). (Kept in memory they would be 4 bytes a
// pair each way, 0.5 GB for 16 windows of 64 tokens over 85,000 keys; the second
// product costs a tenth of that time.) V is never read.
//
// The two are one pipeline on the fifth-generation tensor cores. An item
// holds up to two 128-row tiles X of one operand in shared memory and streams
// 128-row tiles Y of the other past them, S = X . Y^T (tcgen05.mma, M 128, N 128):
//   * kLse: X = (query token, head) rows of a request, Y = its keys; a row's
//     keys may be split over several items (partial log-sum-exps);
//   * kSum: X = keys, Y = query rows, from the first that sees a key;
//   * kWindow, where no request has more than two tiles of rows: X = those
//     rows, Y = keys with S = Y . X^T, so that a key is finished with its tile
//     and K streams past resident rows (with K resident, every 256 keys would
//     stream the rows again: twice the traffic of the product's own).
// A thread then owns one row of an S tile (a tensor-memory lane), so both
// reductions are private to a thread until the item's end.
//   warps 0-15   softmax: group g (four warps, one per scheduler) takes every
//                fourth S tile, warp w its lanes 32 (w mod 4) .. + 31
//   warp 16      issues the MMAs and owns the tensor memory (four S tiles)
//   warp 17      picks the items, streams X (two slots, so the next item's X
//                lands early) and Y
//   warp 18      the query rows' log-sum-exps (kSum, kWindow)
// An S tile costs about 530 clocks of tensor core, 512 of exponentials (32 a
// clock and SM) and 400 issue slots a scheduler at 3 instructions a logit.
#include <cmath>

#include "batch.cuh"
#include "tc.cuh"

namespace mi {
namespace {

constexpr int kLse = 0, kSum = 1, kWindow = 2;
constexpr int kTile = 128;
constexpr int kSoftWarps = 16, kGroups = 4, kMmaWarp = 16, kLoadWarp = 17, kLseWarp = 18;
constexpr int kThreads = 19 * 32;
constexpr int kYSlots = 2, kMaskSlots = 8, kLseSlots = 8, kItemSlots = 4;
constexpr uint32_t kCols = 512;
constexpr int kMergeThreads = 256;

template <int HD>
struct WinSmem {
    static constexpr int kH = HD / 64;
    static constexpr int kT = kH * kTile * 128;          // one tile: kH x [128 rows][128 B], 128-byte swizzle
    static constexpr int kX = 0;                          // [2 slots][2 tiles]
    static constexpr int kY = 4 * kT;                     // [kYSlots]
    static constexpr int kLses = kY + kYSlots * kT;       // [kLseSlots][128] fp32
    static constexpr int kComb = kLses + kLseSlots * kTile * 4;  // [2][kGroups][128] float2
    static constexpr int kItems = kComb + 2 * kGroups * kTile * 8;
    static constexpr int kSums = kItems + kItemSlots * 64;
    static constexpr int kMask = kSums + flat_words(kThreads) * 8;
    static constexpr int kBar = (kMask + kMaskSlots * 4 + 7) / 8 * 8;
    static constexpr int kNBar = 4 + 2 * kYSlots + 2 * kGroups + 2 * kLseSlots + 2 * kItemSlots + 1 + 4;
    static constexpr int kTmem = kBar + kNBar * 8;        // the tensor-memory base, then two words: a wait ran out
    static constexpr int kTotal = kTmem + 16 + 1024;      // slack to align the base to 1024 B
};

struct WindowParams {
    const int32_t* tables;         // [R][mbps]
    const int32_t* lens;           // [R]
    const int32_t* query_start;    // [R + 1]
    float* part;                   // [T][Hq][splits] partial log-sum-exps, base 2
    float* nlse;                   // [Hkv][T][G] the rows' negated log-sum-exps (-inf: no key)
    unsigned int* next;            // [0] kSum: the next item, [1] the key tiles per split (0: bad query_start)
    float* scores;                 // [num_blocks][Hkv][16]
    int32_t* dev_err;
    int R, Hq, Hkv, G, num_blocks, mbps, T, max_q, fresh;
    int xt;                        // kWindow: tiles of rows of every item
    int splits, sms;               // most splits of a row's keys
    float sl2;                     // scale * log2(e), never 0
    long long wait_ns;
    int withhold;                  // failure-detection test: the first Y tile of every block is not announced
};

// Request r: n tokens, the last m of them with queries in rows q0 .. q0+m-1;
// first = n - m (negative: the rows before position 0 see nothing). A request
// with more queries than the call allows has m = -1 and is left alone.
struct Request {
    int n, m, q0, first;
};

__device__ __forceinline__ Request request_of(const WindowParams& p, int r) {
    Request x;
    x.q0 = __ldg(p.query_start + r);
    x.m = __ldg(p.query_start + r + 1) - x.q0;
    x.n = min(max(__ldg(p.lens + r), 0), p.mbps * kBlock);
    x.first = x.n - x.m;
    if (x.m < 0 || x.m > p.max_q) x.m = -1;
    return x;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A Y or X tile of query rows holds whole tokens: tr = (128 / G) * G rows.
__device__ __forceinline__ int row_pairs(const WindowParams& p, const Request& x) {
    const int pr = 2 * (kTile / p.G);  // tokens of two tiles
    return x.m > 0 ? ceil_div(x.m, pr) : 0;
}
// Key tiles that the rows of pair pt see.
__device__ __forceinline__ int seen_tiles(const WindowParams& p, const Request& x, int pt) {
    const int last = x.first + min(x.m, (pt + 1) * 2 * (kTile / p.G)) - 1;
    return last >= 0 ? last / kTile + 1 : 0;
}

// Key tiles per split: about four items per SM, and no more splits of a row
// than the workspace has places for. `most` is a shared word.
__device__ int split_tiles(const WindowParams& p, long long* sums, int* most) {
    const long long total = flat_scan(
        p.R,
        [&](int r) {
            const Request x = request_of(p, r);
            return (long long)p.Hkv * row_pairs(p, x) * ceil_div(x.n, kTile);
        },
        sums);
    if (threadIdx.x == 0) *most = 0;
    __syncthreads();
    int mine = 0;
    for (int r = threadIdx.x; r < p.R; r += blockDim.x) {
        const Request x = request_of(p, r);
        if (x.m > 0) mine = max(mine, ceil_div(x.n, kTile));
    }
    if (mine > 0) atomicMax(most, mine);
    __syncthreads();
    const long long even = (total + 4LL * p.sms - 1) / (4LL * p.sms);
    const int step = max((int)min(even, 1LL << 24), ceil_div(*most, p.splits));
    return max(step, 4);
}

// One work item: X tiles xt (0: the list is over), Y tiles y0 .. y1-1.
struct __align__(16) Item {
    int r, h, xt, y0, y1, row0, split, pad;  // row0: the first query row (kLse) or key (kSum) of X
    Request x;
};
static_assert(sizeof(Item) <= 64, "an item's place in shared memory");

template <int MODE>
__device__ __forceinline__ long long item_count(const WindowParams& p, int r, int step, int xtiles) {
    const Request x = request_of(p, r);
    if (MODE == kLse) return (long long)p.Hkv * row_pairs(p, x) * ceil_div(ceil_div(x.n, kTile), step);
    if (MODE == kWindow) return x.m >= 0 ? (long long)p.Hkv * ceil_div(ceil_div(x.n, kTile), step) : 0ll;
    return x.m >= 0 ? (long long)p.Hkv * ceil_div(x.n, xtiles * kTile) : 0ll;
}

template <int MODE>
__device__ __forceinline__ Item item_at(const WindowParams& p, const long long* sums, long long i, int step,
                                        int xtiles) {
    Item it;
    long long first;
    it.r = flat_find(p.R, [&](int r) { return item_count<MODE>(p, r, step, xtiles); }, sums, i, first);
    it.x = request_of(p, it.r);
    const int o = (int)(i - first), tr = kTile / p.G * p.G, rows = it.x.m * p.G;
    it.h = o % p.Hkv;
    it.split = 0;
    if (MODE == kLse) {
        const int pairs = row_pairs(p, it.x), pt = pairs - 1 - o / p.Hkv % pairs;  // the longest first
        it.split = o / p.Hkv / pairs;
        it.row0 = pt * 2 * tr;
        it.xt = rows - it.row0 > tr ? 2 : 1;
        it.y0 = it.split * step;
        it.y1 = min(it.y0 + step, seen_tiles(p, it.x, pt));
    } else if (MODE == kWindow) {
        it.row0 = 0;
        it.xt = p.xt;
        it.y0 = o / p.Hkv * step;
        it.y1 = min(it.y0 + step, ceil_div(it.x.n, kTile));
    } else {
        it.row0 = o / p.Hkv * xtiles * kTile;
        it.xt = min(xtiles, ceil_div(it.x.n - it.row0, kTile));
        it.y0 = max(0, it.row0 - it.x.first) * p.G / tr;  // rows before it see none of the keys
        it.y1 = max(it.y0, ceil_div(rows, tr));
    }
    return it;
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, long long limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit_ns, kWaitSleepNs));
}

template <int HD, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const WindowParams p) {
    using SM = WinSmem<HD>;
    constexpr int kH = SM::kH;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    unsigned char* base = smem_raw + (sbase - raw);
    long long* sums = reinterpret_cast<long long*>(base + SM::kSums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sbase + SM::kBar;
    const uint32_t x_full = bar, x_empty = bar + 16, y_full = bar + 32, y_empty = y_full + 8 * kYSlots;
    const uint32_t s_full = y_empty + 8 * kYSlots, s_empty = s_full + 8 * kGroups;
    const uint32_t l_full = s_empty + 8 * kGroups, l_empty = l_full + 8 * kLseSlots;
    const uint32_t i_full = l_empty + 8 * kLseSlots, i_empty = i_full + 8 * kItemSlots, fin = i_empty + 8 * kItemSlots;
    const uint32_t c_full = fin + 8;  // kWindow: [2 pairs of groups][2] the second group's sums
    volatile int* failed = reinterpret_cast<volatile int*>(base + SM::kTmem + 4);
    const uint32_t mask0 = sbase + SM::kMask;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(x_full + 8 * i, 1);
            mbar_init(x_empty + 8 * i, 1);
        }
        for (int i = 0; i < kYSlots; ++i) {
            mbar_init(y_full + 8 * i, 1);
            mbar_init(y_empty + 8 * i, 1);
        }
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(s_full + 8 * i, 2);   // the MMAs' commit, and the issuing warp (for what it has seen)
            mbar_init(s_empty + 8 * i, 4);  // the warps of a group
        }
        for (int i = 0; i < kLseSlots; ++i) {
            mbar_init(l_full + 8 * i, 32);  // the copying lanes
            mbar_init(l_empty + 8 * i, kSoftWarps);
        }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(i_full + 8 * i, 1);
            mbar_init(i_empty + 8 * i, kSoftWarps + 1 + (MODE != kLse ? 1 : 0));  // every warp that reads items
        }
        mbar_init(fin, 1);
        for (int i = 0; i < 4; ++i) mbar_init(c_full + 8 * i, 4);
        failed[0] = failed[1] = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::alloc(sbase + SM::kTmem, kCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tbase = lds32(sbase + SM::kTmem);
    pdl_wait();
    pdl_trigger();

    // ---------------------------------------------------------- the plan --
    long long total = 0;
    int step = 0, xtiles = 2;
    if (MODE == kLse) {
        const bool ascend = starts_ascend(p.query_start, p.R, p.T);
        const int g = blockIdx.x * kThreads + threadIdx.x;
        if (!ascend && g == 0) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
        for (int r = g; ascend && r < p.R; r += gridDim.x * kThreads) {
            const Request x = request_of(p, r);
            if (x.m < 0 || x.m > x.n) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
            if (__ldg(p.lens + r) > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
        }
        if (ascend) step = split_tiles(p, sums, reinterpret_cast<int*>(base + SM::kMask));
        if (g == 0) p.next[1] = (unsigned int)step;
    } else {
        step = (int)__ldcg(p.next + 1);
    }
    if (step > 0) {
        auto items = [&](int r) { return item_count<MODE>(p, r, step, xtiles); };
        total = flat_scan(p.R, items, sums);
        if (MODE == kSum && total < 4LL * p.sms) {
            // single tiles of keys while pairs would leave SMs with few
            xtiles = 1;
            __syncthreads();
            total = flat_scan(p.R, items, sums);
        }
    }
    const int tr = kTile / p.G * p.G;
    // the k-th item of the list as every other warp sees it
    auto take = [&](uint32_t k, Item& it) -> bool {
        const uint32_t sl = k % kItemSlots;
        if (!wait_warp(i_full + 8 * sl, (k / kItemSlots) & 1, p.wait_ns)) return false;
        it = *reinterpret_cast<const Item*>(base + SM::kItems + sl * 64);
        __syncwarp();
        if (lane == 0) mbar_arrive(i_empty + 8 * sl);
        return true;
    };

    if (warp == kLoadWarp) {
        // ------------------------------------------------------- loads ----
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        uint32_t xc = 0, yc = 0;
        bool ok = true;
        // the lane's block of key tiles j .. j + tiles - 1 (-1: none; -2: not in the cache)
        auto entry = [&](const Item& it, int j, int tiles) -> int {
            const int x = j * (kTile / kBlock) + lane;
            if (lane >= tiles * (kTile / kBlock) || x * kBlock >= it.x.n) return -1;
            const int blk = __ldg(p.tables + (long long)it.r * p.mbps + x);
            return blk >= 0 && blk < p.num_blocks ? blk : -2;
        };
        // those blocks to dst, each as kH 64-column halves; kLse posts the
        // tile's mask of blocks in the cache
        auto load_keys = [&](const Item& it, uint32_t dst, uint32_t fb, int blk) {
            if (MODE == kLse && blk == -2) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
            const uint32_t msk = __ballot_sync(0xffffffffu, blk >= 0);
            if (lane == 0) {
                if (MODE == kLse) sts32(mask0 + (yc % kMaskSlots) * 4, msk);
                mbar_arrive_expect_tx(fb, (uint32_t)__popc(msk) * kH * kBlock * 128u);
            }
            __syncwarp();
            if (blk >= 0) {
                const uint32_t kd = dst + (lane >> 3) * SM::kT + (lane & 7) * kBlock * 128;
                const int row0 = (blk * p.Hkv + it.h) * kBlock;
                for (int hh = 0; hh < kH; ++hh) tma_load_3d(kd + hh * kTile * 128, &tmk, fb, 0, hh, row0, policy);
            }
        };
        auto load_rows = [&](const Item& it, uint32_t dst, uint32_t fb, int row0, int tiles) {
            if (lane == 0) {
                mbar_arrive_expect_tx(fb, (uint32_t)(tiles * kH * tr) * 128u);
                for (int t = 0; t < tiles; ++t)
                    for (int hh = 0; hh < kH; ++hh)
                        tma_load_4d(dst + t * SM::kT + hh * kTile * 128, &tmq, fb, 0, hh, it.h * p.G,
                                    it.x.q0 + row0 / p.G + t * (tr / p.G), policy);
            }
            __syncwarp();
        };
        // kLse and kWindow deal the list out back and forth (it goes from long
        // to short); kSum's items are taken from a counter as blocks get free
        auto pick = [&](long long k) -> long long {
            if (MODE != kSum) return k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            unsigned int i = 0;
            if (lane == 0) i = atomicAdd(p.next, 1u);
            return (long long)__shfl_sync(0xffffffffu, i, 0);
        };
        long long k = 0, i = pick(0);
        uint32_t ic = 0;
        for (;;) {
            Item it;
            it.xt = 0;
            if (i < total) {
                it = item_at<MODE>(p, sums, i, step, xtiles);
                if (MODE == kLse && it.y0 >= it.y1) {  // keys past what the rows see
                    i = pick(++k);
                    continue;
                }
            }
            const uint32_t sl = ic % kItemSlots;
            if (!(ok = wait_warp(i_empty + 8 * sl, ((ic / kItemSlots) & 1) ^ 1, p.wait_ns))) break;
            if (lane == 0) {
                *reinterpret_cast<Item*>(base + SM::kItems + sl * 64) = it;
                mbar_arrive(i_full + 8 * sl);
            }
            __syncwarp();
            ++ic;
            if (it.xt == 0) break;
            i = pick(++k);
            if (it.y0 >= it.y1) continue;
            const uint32_t xs = xc & 1;
            if (!(ok = wait_warp(x_empty + 8 * xs, ((xc >> 1) & 1) ^ 1, p.wait_ns))) break;
            const uint32_t xd = sbase + SM::kX + xs * 2 * SM::kT;
            if (MODE == kSum)
                load_keys(it, xd, x_full + 8 * xs, entry(it, it.row0 / kTile, it.xt));
            else
                load_rows(it, xd, x_full + 8 * xs, it.row0, it.xt);
            ++xc;
            // table entries are read a tile ahead of their use
            int blk = MODE == kSum ? 0 : entry(it, it.y0, 1);
            for (int j = it.y0; j < it.y1; ++j, ++yc) {
                const int now = blk;
                if (MODE != kSum && j + 1 < it.y1) blk = entry(it, j + 1, 1);
                const uint32_t ys = yc % kYSlots;
                if (!(ok = wait_warp(y_empty + 8 * ys, ((yc / kYSlots) & 1) ^ 1, p.wait_ns))) break;
                if (p.withhold && yc == 0) continue;
                const uint32_t yd = sbase + SM::kY + ys * SM::kT;
                if (MODE == kSum)
                    load_rows(it, yd, y_full + 8 * ys, j * tr, 1);
                else
                    load_keys(it, yd, y_full + 8 * ys, now);
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
            // copies issued land before the block's shared memory goes away
            for (uint32_t s = 0; s < 2; ++s)
                if (xc > s) (void)wait_warp(x_full + 8 * s, ((xc - 1 - s) / 2) & 1, drain_limit(p.wait_ns));
            for (uint32_t s = p.withhold ? 1 : 0; s < kYSlots; ++s)
                if (yc > s) (void)wait_warp(y_full + 8 * s, ((yc - 1 - s) / kYSlots) & 1, drain_limit(p.wait_ns));
        }
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------- MMA issuer ----
        constexpr uint32_t id = tc::idesc_bf16(kTile, kTile, false);
        uint32_t xc = 0, yc = 0, sc = 0;
        bool ok = true;
        for (uint32_t ic = 0; ok; ++ic) {
            Item it;
            if (!(ok = take(ic, it)) || it.xt == 0) break;
            if (it.y0 >= it.y1) continue;
            if (!(ok = wait_warp(x_full + 8 * (xc & 1), (xc >> 1) & 1, p.wait_ns))) break;
            for (int j = it.y0; ok && j < it.y1; ++j, ++yc) {
                if (!(ok = wait_warp(y_full + 8 * (yc % kYSlots), (yc / kYSlots) & 1, p.wait_ns))) break;
                const uint32_t ya = sbase + SM::kY + (yc % kYSlots) * SM::kT;
                for (int t = 0; t < it.xt; ++t, ++sc) {
                    const uint32_t b = sc % kGroups;
                    if (!(ok = wait_warp(s_empty + 8 * b, ((sc / kGroups) & 1) ^ 1, p.wait_ns))) break;
                    tc::fence_after();
                    const uint32_t xa = sbase + SM::kX + ((xc & 1) * 2 + t) * SM::kT;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kTile * 128 + (kk & 3) * 32;
                        const uint64_t xd = tc::sdesc_sw128(xa + off, 16, 1024), yd = tc::sdesc_sw128(ya + off, 16, 1024);
                        tc::mma_ss_elect(tbase + b * kTile, MODE == kWindow ? yd : xd, MODE == kWindow ? xd : yd, id,
                                         kk > 0);
                    }
                    tc::commit_elect(s_full + 8 * b);
                    if (lane == 0) mbar_arrive(s_full + 8 * b);
                    __syncwarp();
                }
                if (ok) tc::commit_elect(y_empty + 8 * (yc % kYSlots));
            }
            if (ok) tc::commit_elect(x_empty + 8 * (xc & 1));
            ++xc;
        }
        if (!ok && lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
        // every MMA issued has finished before tensor memory is released
        tc::commit_elect(fin);
        (void)wait_warp(fin, 0, drain_limit(p.wait_ns));
    } else if (warp == kLseWarp) {
        if (MODE != kLse) {
            // -------------------------------- the rows' log-sum-exps ----
            // Copied without a wait, so the ring is filled ahead; zero past a
            // tile's rows. kSum: one slot per Y tile; kWindow: two per item,
            // its X tiles.
            uint32_t lc = 0;
            bool ok = true;
            for (uint32_t ic = 0; ok; ++ic) {
                Item it;
                if (!(ok = take(ic, it)) || it.xt == 0) break;
                const int rows = it.x.m * p.G;
                const float* at = p.nlse + ((long long)it.h * p.T + it.x.q0) * p.G;
                const int j0 = MODE == kSum ? it.y0 : 0, j1 = MODE == kSum ? it.y1 : 2;
                for (int j = j0; j < j1; ++j, ++lc) {
                    const uint32_t ls = lc % kLseSlots;
                    if (!(ok = wait_warp(l_empty + 8 * ls, ((lc / kLseSlots) & 1) ^ 1, p.wait_ns))) break;
#pragma unroll
                    for (int u = 0; u < kTile / 32; ++u) {
                        const int c = u * 32 + lane, rho = j * tr + c;
                        const bool in = c < tr && rho < rows;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                         sbase + SM::kLses + (ls * kTile + c) * 4),
                                     "l"(in ? at + rho : p.nlse), "r"(in ? 4 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(l_full + 8 * ls) : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (!ok && lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
        }
    } else {
        // ---------------------------------------------------- softmax ----
        const int group = warp >> 2, quad = warp & 3;
        const int my = quad * 32 + lane;  // row of a tile, tensor-memory lane
        const uint32_t ts = tbase + ((uint32_t)(quad * 32) << 16) + (uint32_t)(group * kTile);
        const uint64_t sc2 = tc::f2(p.sl2, p.sl2);
        const bool pos_scale = p.sl2 > 0.f;
        const float off_value = pos_scale ? -INFINITY : INFINITY;  // a masked logit, before the scale
        uint32_t yc = 0, sc = 0, wc = 0;
        bool ok = true;
        for (uint32_t ic = 0;; ++ic) {
            Item it;
            if (!take(ic, it)) {
                ok = false;
                it.xt = 1;
                it.y0 = it.y1 = 0;
                it.x.m = it.x.n = 0;
            }
            if (it.xt == 0) break;
            const int rows = it.x.m * p.G;
            // kLse: the last key this thread's row sees; kSum: the first row
            // that sees this thread's key
            const int tile = it.xt == 2 ? (group ^ (int)sc) & 1 : 0;  // this group's S tiles of the item
            int bound = 0;
            bool mine = false;
            if (MODE == kLse) {
                const int rho = it.row0 + tile * tr + my;
                mine = my < tr && rho < rows;
                bound = mine ? it.x.first + rho / p.G : 0x3FFFFFFF;
            } else if (MODE == kSum) {
                const int t = it.row0 + tile * kTile + my;
                mine = t < it.x.n;
                bound = mine ? max(0, t - it.x.first) * p.G : 0;
            }
            float m = -INFINITY, total_sum = 0.f;  // kLse: the sum is relative to 2^m
            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
            // f(x, q) for the S tile's four chunks of 32 columns, the next one
            // loaded under the arithmetic of the one at hand; stops after
            // `cols` columns
            auto sweep = [&](int cols, auto f) {
                uint32_t xa[32], xb[32];
                tc::ld32(ts, xa);
#pragma unroll 1
                for (int q = 0; q < 4; q += 2) {
                    tc::wait_ld();
                    tc::ld32(ts + 32u * q + 32u, xb);
                    f(xa, q);
                    tc::wait_ld();
                    const bool more = 32 * q + 64 < cols;
                    if (q == 0 && more) tc::ld32(ts + 64u, xa);
                    if (32 * q + 32 < cols) f(xb, q + 1);
                    if (!more) break;
                }
            };
            // columns lo .. hi - 1 of a chunk count
            auto cut = [&](uint32_t (&x)[32], int lo, int hi) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < lo || c >= hi) x[c] = __float_as_uint(off_value);
            };
            if (MODE == kWindow)
                ok = ok && wait_warp(l_full + 8 * (2 * ic % kLseSlots), (2 * ic / kLseSlots) & 1, p.wait_ns) &&
                     wait_warp(l_full + 8 * ((2 * ic + 1) % kLseSlots), (2 * ic / kLseSlots) & 1, p.wait_ns);
            for (int j = it.y0; ok && j < it.y1; ++j, ++yc) {
                if (MODE == kSum &&
                    !(ok = wait_warp(l_full + 8 * (yc % kLseSlots), (yc / kLseSlots) & 1, p.wait_ns)))
                    break;
                const int key = j * kTile + my;  // kWindow: this thread's key of the stage, its block and row there
                int blk = -1;
                // this group's S tile of the stage, if it has one
                const int t = (group - (int)sc) & (kGroups - 1);
                if (t < it.xt) {
                    if (!(ok = wait_warp(s_full + 8 * group, ((sc + t) / kGroups) & 1, p.wait_ns))) break;
                    tc::fence_after();
                    if (MODE == kLse) {
                        const uint32_t msk = lds32(mask0 + (yc % kMaskSlots) * 4);
                        const bool part = __any_sync(0xffffffffu, msk != 0xFFu || j * kTile + kTile - 1 > bound);
                        auto mask = [&](uint32_t (&x)[32], int q) {
                            if (!part) return;
                            const uint32_t have = (msk >> (2 * q)) & 3u;
                            const int hi = bound - (j * kTile + 32 * q) + 1;
                            cut(x, have & 1u ? 0 : 16, have & 2u ? hi : min(hi, 16));
                        };
                        // The sum is relative to m, the largest of the first
                        // tile's logits: fp32 holds it however far later ones
                        // lie below, and above until it nears overflow. Only
                        // then, and at first, is a maximum taken and the sum
                        // moved to it.
                        bool top = __any_sync(0xffffffffu, m == -INFINITY);
                        for (;;) {
                            if (top) {
                                float e4[4] = {off_value, off_value, off_value, off_value};
                                sweep(kTile, [&](uint32_t (&x)[32], int q) {
                                    mask(x, q);
#pragma unroll
                                    for (int c = 0; c < 32; ++c)
                                        e4[c & 3] = pos_scale ? fmaxf(e4[c & 3], __uint_as_float(x[c]))
                                                              : fminf(e4[c & 3], __uint_as_float(x[c]));
                                });
                                const float best = (pos_scale ? fmaxf(fmaxf(e4[0], e4[1]), fmaxf(e4[2], e4[3]))
                                                              : fminf(fminf(e4[0], e4[1]), fminf(e4[2], e4[3]))) * p.sl2;
                                total_sum *= best > m ? ex2(m - best) : 1.f;
                                m = fmaxf(m, best);
                            }
                            const float nu = m == -INFINITY ? 0.f : -m;
                            const uint64_t nu2 = tc::f2(nu, nu);
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[c] = 0ull;
                            sweep(kTile, [&](uint32_t (&x)[32], int q) {
                                mask(x, q);
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    const uint64_t a = tc::fma2(tc::f2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, nu2);
                                    acc[c & 3] = tc::add2(acc[c & 3], tc::f2(ex2(tc::f2_lo(a)), ex2(tc::f2_hi(a))));
                                }
                            });
                            const uint64_t a2 = tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3]));
                            const float now = total_sum + (tc::f2_lo(a2) + tc::f2_hi(a2));
                            if (top || !__any_sync(0xffffffffu, now > 0x1p100f)) {
                                total_sum = now;
                                break;
                            }
                            top = true;
                        }
                    } else {
                        // the Y rows of kSum, the X rows of kWindow: columns
                        // from `first` on see the thread's key, `cols` hold rows
                        const int row0 = (MODE == kSum ? j : tile) * tr, cols = min(tr, rows - row0);
                        if (MODE == kWindow) {
                            if (t == 0 && key < it.x.n) blk = __ldg(p.tables + (long long)it.r * p.mbps + key / kBlock);
                            bound = (key - it.x.first) * p.G;
                        }
                        const int first = bound - row0;
                        const bool part = __any_sync(0xffffffffu, first > 0) || (cols & 31) != 0;
                        const uint32_t la = sbase + SM::kLses + ((MODE == kSum ? yc : 2 * ic + tile) % kLseSlots) * kTile * 4;
                        if (MODE == kWindow) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[c] = 0ull;
                        }
                        if (cols > 0)
                            sweep(cols, [&](uint32_t (&x)[32], int q) {
                                if (part) cut(x, first - 32 * q, cols - 32 * q);
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    uint32_t l0, l1, l2, l3;
                                    lds128(la + 128 * q + 16 * c, l0, l1, l2, l3);
                                    const uint64_t a0 = tc::fma2(tc::f2(__uint_as_float(x[4 * c]), __uint_as_float(x[4 * c + 1])), sc2,
                                                                 tc::f2(__uint_as_float(l0), __uint_as_float(l1)));
                                    const uint64_t a1 = tc::fma2(tc::f2(__uint_as_float(x[4 * c + 2]), __uint_as_float(x[4 * c + 3])), sc2,
                                                                 tc::f2(__uint_as_float(l2), __uint_as_float(l3)));
                                    acc[(2 * c) & 3] = tc::add2(acc[(2 * c) & 3], tc::f2(ex2(tc::f2_lo(a0)), ex2(tc::f2_hi(a0))));
                                    acc[(2 * c + 1) & 3] = tc::add2(acc[(2 * c + 1) & 3], tc::f2(ex2(tc::f2_lo(a1)), ex2(tc::f2_hi(a1))));
                                }
                            });
                    }
                    // the tile has been read: hand it back
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty + 8 * group);
                    if (MODE == kWindow) {
                        // the second tile's group hands its sums to the first's
                        // through one of two places (the first group's S tile of
                        // two stages on waits for it to be done with this one)
                        const uint64_t a = tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3]));
                        float w = tc::f2_lo(a) + tc::f2_hi(a);
                        const int place = (group & 2) + (int)(wc & 1);
                        float* comb = reinterpret_cast<float*>(base + SM::kComb) + place * kTile;
                        if (t == 1) {
                            comb[my] = w;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(c_full + 8 * place);
                        } else {
                            if (it.xt == 2) {
                                if (!(ok = wait_warp(c_full + 8 * place, (wc >> 1) & 1, p.wait_ns))) break;
                                w += comb[my];
                            }
                            if (blk >= 0 && blk < p.num_blocks) {
                                float* at = p.scores + ((long long)blk * p.Hkv + it.h) * kBlock + key % kBlock;
                                *at = p.fresh || key >= it.x.first ? w : *at + w;
                            }
                        }
                        ++wc;
                    }
                }
                sc += it.xt;
                if (MODE == kSum) {
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(l_empty + 8 * (yc % kLseSlots));
                }
            }
            if (MODE == kWindow) {
                if (!ok) break;
                __syncwarp();
                if (lane < 2) mbar_arrive(l_empty + 8 * ((2 * ic + lane) % kLseSlots));
                continue;
            }
            // the groups that share a row: every second one, or all four for a
            // single tile. A warp whose wait ran out still meets the others
            // here, and all of them leave together.
            float sum = total_sum;
            if (MODE == kSum) {
                const uint64_t a = tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3]));
                sum = tc::f2_lo(a) + tc::f2_hi(a);
            }
            float2* comb = reinterpret_cast<float2*>(base + SM::kComb) + (ic & 1) * kGroups * kTile;
            if (!ok && lane == 0) failed[ic & 1] = 1;
            comb[group * kTile + my] = make_float2(m, sum);
            asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
            if (failed[ic & 1]) {
                ok = false;
                break;
            }
            if (mine && group < it.xt) {
                float2 q[4];
                const int parts = it.xt == 2 ? 2 : 4;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    q[u] = u < parts ? comb[(it.xt == 2 ? u * 2 + group : u) * kTile + my] : make_float2(-INFINITY, 0.f);
                if (MODE == kLse) {
                    const float M = fmaxf(fmaxf(q[0].x, q[1].x), fmaxf(q[2].x, q[3].x));
                    const float v = M == -INFINITY ? 0.f : M;
                    const float l = (q[0].y * exp2f(q[0].x - v) + q[1].y * exp2f(q[1].x - v)) +
                                    (q[2].y * exp2f(q[2].x - v) + q[3].y * exp2f(q[3].x - v));
                    const int rho = it.row0 + tile * tr + my;
                    p.part[((long long)(it.x.q0 + rho / p.G) * p.Hq + (long long)it.h * p.G + rho % p.G) * p.splits + it.split] =
                        l == 0.f ? -INFINITY : M + log2f(l);
                } else {
                    const float w = (q[0].y + q[1].y) + (q[2].y + q[3].y);
                    const int t = it.row0 + tile * kTile + my;
                    const int blk = __ldg(p.tables + (long long)it.r * p.mbps + t / kBlock);
                    if (blk >= 0 && blk < p.num_blocks) {
                        float* at = p.scores + ((long long)blk * p.Hkv + it.h) * kBlock + t % kBlock;
                        *at = p.fresh || t >= it.x.first ? w : *at + w;
                    }
                }
            }
        }
        if (!ok && lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::dealloc(tbase, kCols);
    }
}

// Each row's log-sum-exp from its splits (one launch between the two: the
// second reads every row once per 256 keys), and kSum's item counter back to
// zero. A thread merges one row.
__global__ void __launch_bounds__(kMergeThreads) window_merge_kernel(const WindowParams p) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.next = 0u;
    const int step = (int)__ldcg(p.next + 1);
    if (step == 0) return;
    const long long row = (long long)blockIdx.x * kMergeThreads + threadIdx.x;
    const int i = (int)(row / p.Hq);
    if (i < __ldg(p.query_start) || i >= __ldg(p.query_start + p.R)) return;
    int lo = 0, hi = p.R;  // query_start[lo] <= i < query_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.query_start + mid) <= i) lo = mid;
        else hi = mid;
    }
    const Request x = request_of(p, lo);
    if (x.m < 0) return;
    const int n = ceil_div(seen_tiles(p, x, (i - x.q0) / (2 * (kTile / p.G))), step);
    const float* at = p.part + row * p.splits;
    float M = -INFINITY, sum = 0.f;
#pragma unroll 8
    for (int s = 0; s < n; ++s) M = fmaxf(M, __ldcg(at + s));
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
        const float v = __ldcg(at + s);
        sum += v == -INFINITY ? 0.f : exp2f(v - M);
    }
    p.nlse[((long long)(row % p.Hq / p.G) * p.T + i) * p.G + row % p.G] = sum == 0.f ? -INFINITY : -(M + log2f(sum));
}

// Places for partial log-sum-exps per row: enough splits that few row tiles
// still fill the GPU, fewer where the rows themselves are many.
int split_places(const mi_dims& D, int32_t total_q) {
    const long long rows = (long long)total_q * D.Hq;
    return rows <= (1LL << 20) ? 32 : rows <= (1LL << 23) ? 8 : 2;
}

size_t lse_bytes(const mi_dims& D, int32_t total_q) { return ((size_t)total_q * D.Hq * 4 + 255) / 256 * 256; }

size_t window_bytes(const mi_dims& D, int32_t total_q) {
    return lse_bytes(D, total_q) * (1 + split_places(D, total_q)) + 256;
}

bool window_sizes_ok(const mi_dims& D, int32_t total_q, int32_t max_query_len) {
    return total_q >= 0 && max_query_len >= 0 && (long long)total_q * D.Hq <= 0x7FFFFFFFLL &&
           (long long)max_query_len * D.Hq <= 0x7FFFFFFFLL;
}

template <int HD, int MODE>
bool launch_window(const CUtensorMap& tq, const CUtensorMap& tk, const WindowParams& p, cudaStream_t st) {
    static std::mutex mu;
    static CUcontext done[256] = {};
    if (!raise_smem(reinterpret_cast<const void*>(window_kernel<HD, MODE>), WinSmem<HD>::kTotal, done, mu)) return false;
    return launch_pdl(window_kernel<HD, MODE>, p.sms, kThreads, WinSmem<HD>::kTotal, st, tq, tk, p) == cudaSuccess;
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_paged_prefill_scores_workspace_bytes(const mi_dims* dims, int32_t total_q, int32_t max_query_len) {
    using namespace mi;
    if (check_paged_dims(dims) != MI_OK || !window_sizes_ok(*dims, total_q, max_query_len)) return 0;
    return window_bytes(*dims, total_q);
}

extern "C" mi_status mi_paged_prefill_scores(const mi_dims* dims, int32_t total_q, int32_t max_query_len,
                                             const void* q, const void* k_cache, const int32_t* block_tables,
                                             const int32_t* context_lens, const int32_t* query_start, float scale,
                                             int32_t fresh, float* scores, void* workspace, size_t workspace_bytes,
                                             int32_t* dev_err, mi_stream_t stream) {
    using namespace mi;
    const mi_status ds = check_paged_dims(dims);
    if (ds != MI_OK) return ds;
    const mi_dims D = *dims;
    if (!window_sizes_ok(D, total_q, max_query_len) || !std::isfinite(scale)) return MI_ERR_INVALID_ARG;
    if (D.B == 0) return MI_OK;
    if (!k_cache || !block_tables || !context_lens || !query_start || !scores || !workspace || (total_q > 0 && !q))
        return MI_ERR_INVALID_ARG;
    if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(scores, 16) || !aligned_to(workspace, 16))
        return MI_ERR_INVALID_ARG;
    if (workspace_bytes < window_bytes(D, total_q)) return MI_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return MI_ERR_CUDA;
    const int G = D.Hq / D.Hkv, HD = D.head_dim;
    WindowParams p;
    p.tables = block_tables;
    p.lens = context_lens;
    p.query_start = query_start;
    p.next = static_cast<unsigned int*>(workspace);
    p.nlse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256 + lse_bytes(D, total_q));
    p.scores = scores;
    p.dev_err = dev_err;
    p.R = D.B;
    p.Hq = D.Hq;
    p.Hkv = D.Hkv;
    p.G = G;
    p.num_blocks = D.num_blocks;
    p.mbps = D.max_blocks_per_seq;
    p.T = total_q;
    p.max_q = max_query_len;
    p.fresh = fresh != 0;
    p.xt = 0;
    p.splits = split_places(D, total_q);
    p.sms = sms;
    p.sl2 = scale * 1.4426950408889634f;
    // a scale of 0 weighs every key the same, and so does one that leaves
    // every logit far below 2^-24 (a masked logit times 0 would be NaN)
    if (p.sl2 == 0.f) p.sl2 = 1.2e-38f;
    p.wait_ns = test_wait_limit_ns();
    p.withhold = test_withhold_copy() ? 1 : 0;
    CUtensorMap tq, tk;
    // without queries nothing is loaded through the first map; it may name any tensor
    if (!make_tmap_q_group(&tq, total_q > 0 ? q : k_cache, total_q > 0 ? total_q : 1, D.Hq, HD, G, kTile / G * G) ||
        !make_tmap_kv_halves(&tk, k_cache, (long long)D.num_blocks * D.Hkv * kBlock, HD))
        return MI_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const long long rows = (long long)total_q * D.Hq;
    const bool wide = HD == 128;
    bool ok = wide ? launch_window<128, kLse>(tq, tk, p, st) : launch_window<64, kLse>(tq, tk, p, st);
    if (ok)
        ok = launch_pdl(window_merge_kernel, (int)((rows + kMergeThreads) / kMergeThreads), kMergeThreads, 0, st, p) ==
             cudaSuccess;
    // rows that fit in two tiles stay resident while the keys stream
    const int tr = kTile / G * G;
    const bool few = (long long)max_query_len * G <= 2 * tr;
    p.xt = max_query_len * G <= tr ? 1 : 2;
    if (ok && few) ok = wide ? launch_window<128, kWindow>(tq, tk, p, st) : launch_window<64, kWindow>(tq, tk, p, st);
    if (ok && !few) ok = wide ? launch_window<128, kSum>(tq, tk, p, st) : launch_window<64, kSum>(tq, tk, p, st);
    return ok ? MI_OK : MI_ERR_CUDA;
}
