// mi_paged_prefill_scores: the attention weight every cached token receives
// from many query tokens at once (the last tokens of a prompt, or all of it).
//
//   score[r][h][t] (+)= sum over query tokens i of request r with t <= pos_i
//                       and the G query heads j of h of 2^(x_ijt - lse_ij)
//
// A weight needs its row's log-sum-exp over all keys, so the logits x are
// computed twice: the first launch reduces them over the keys of each row, the
// second over the rows of each key. (Kept in memory they would be 4 bytes a
// pair each way, 0.5 GB for 16 windows of 64 tokens over 85,000 keys; the second
// product costs a tenth of that time.) V is never read.
//
// Both launches are one pipeline on the fifth-generation tensor cores. An item
// holds up to two 128-row tiles X of one operand in shared memory and streams
// 128-row tiles Y of the other past them, S = X . Y^T (tcgen05.mma, M 128, N 128):
//   * kLse: X = (query token, head) rows of a request, Y = its keys; a row's
//     keys may be split over several items (partial log-sum-exps);
//   * kSum: X = keys, Y = query rows, from the first that sees a key.
// A thread then owns one row of S (a tensor-memory lane) and half its columns,
// so both reductions are private to a thread until the item's end.
//   warps 0-15   softmax: group (warp / 8) takes every second S tile; warp w
//                reads lanes 32 (w mod 4) .. + 31, columns 64 (w / 4 mod 2) .. + 63
//   warp 16      issues the MMAs and owns the tensor memory (four S tiles)
//   warp 17      streams X (two slots, so the next item's X lands early) and Y
//   warp 18      kSum: the Y rows' log-sum-exps, merged from their splits
// The exponentials bound both launches: 16 a clock and SM, against 28 pairs a
// clock for the product.
#include <cmath>

#include "batch.cuh"
#include "tc.cuh"

namespace mi {
namespace {

constexpr int kLse = 0, kSum = 1;
constexpr int kTile = 128;
constexpr int kSoftWarps = 16, kMmaWarp = 16, kLoadWarp = 17, kLseWarp = 18;
constexpr int kThreads = 19 * 32;
constexpr int kYSlots = 2, kSBufs = 4, kMaskSlots = 8, kLseSlots = 4;
constexpr uint32_t kCols = 512;

template <int HD>
struct WinSmem {
    static constexpr int kH = HD / 64;
    static constexpr int kT = kH * kTile * 128;          // one tile: kH x [128 rows][128 B], 128-byte swizzle
    static constexpr int kX = 0;                          // [2 slots][2 tiles]
    static constexpr int kY = 4 * kT;                     // [kYSlots]
    static constexpr int kLses = kY + kYSlots * kT;       // [kLseSlots][128] fp32
    static constexpr int kComb = kLses + kLseSlots * kTile * 4;  // [2][2][2][128] float2
    static constexpr int kSums = kComb + 8 * kTile * 8;
    static constexpr int kMask = kSums + flat_words(kThreads) * 8;
    static constexpr int kBar = (kMask + kMaskSlots * 4 + 7) / 8 * 8;
    static constexpr int kNBar = 4 + 2 * kYSlots + 2 * kSBufs + 2 * kLseSlots + 1;
    static constexpr int kTmem = kBar + kNBar * 8;        // the tensor-memory base, then two words: a wait ran out
    static constexpr int kTotal = kTmem + 16 + 1024;      // slack to align the base to 1024 B
};

struct WindowParams {
    const int32_t* tables;         // [R][mbps]
    const int32_t* lens;           // [R]
    const int32_t* query_start;    // [R + 1]
    float* part;                   // [T][Hq][splits] partial log-sum-exps, base 2
    float* scores;                 // [num_blocks][Hkv][16]
    int32_t* dev_err;
    int R, Hq, Hkv, G, num_blocks, mbps, T, max_q, fresh;
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

// Key tiles per split, the same in every block of both launches: about eight
// items per SM, and no more splits of a row than the workspace has places for.
__device__ int split_tiles(const WindowParams& p, long long* sums, int* shared_max) {
    const long long total = flat_scan(
        p.R,
        [&](int r) {
            const Request x = request_of(p, r);
            return (long long)p.Hkv * row_pairs(p, x) * ceil_div(x.n, kTile);
        },
        sums);
    int most = 0;
    for (int r = threadIdx.x; r < p.R; r += blockDim.x) {
        const Request x = request_of(p, r);
        if (x.m > 0) most = max(most, ceil_div(x.n, kTile));
    }
    if (threadIdx.x == 0) *shared_max = 0;
    __syncthreads();
    if (most > 0) atomicMax(shared_max, most);
    __syncthreads();
    const long long even = (total + 8LL * p.sms - 1) / (8LL * p.sms);
    const int step = max((int)min(even, 1LL << 24), ceil_div(*shared_max, p.splits));
    return max(step, 4);
}

// One work item: X tiles xt (0: nothing to do), Y tiles y0 .. y1-1.
struct Item {
    int r, h, xt, y0, y1, row0, split;  // row0: the first query row (kLse) or key (kSum) of X
    Request x;
};

template <int MODE>
__device__ __forceinline__ long long item_count(const WindowParams& p, int r, int step, int xtiles) {
    const Request x = request_of(p, r);
    if (MODE == kLse) return (long long)p.Hkv * row_pairs(p, x) * ceil_div(ceil_div(x.n, kTile), step);
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
        const int pairs = row_pairs(p, it.x), pt = o / p.Hkv % pairs;
        it.split = o / p.Hkv / pairs;
        it.row0 = pt * 2 * tr;
        it.xt = rows - it.row0 > tr ? 2 : 1;
        it.y0 = it.split * step;
        it.y1 = min(it.y0 + step, seen_tiles(p, it.x, pt));
        if (it.y0 >= it.y1) it.xt = 0;
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
    float* lses = reinterpret_cast<float*>(base + SM::kLses);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sbase + SM::kBar;
    const uint32_t x_full = bar, x_empty = bar + 16, y_full = bar + 32, y_empty = y_full + 8 * kYSlots;
    const uint32_t s_full = y_empty + 8 * kYSlots, s_empty = s_full + 8 * kSBufs;
    const uint32_t l_full = s_empty + 8 * kSBufs, l_empty = l_full + 8 * kLseSlots, fin = l_empty + 8 * kLseSlots;
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
        for (int i = 0; i < kSBufs; ++i) {
            mbar_init(s_full + 8 * i, 2);   // the MMAs' commit, and the issuing warp (for what it has seen)
            mbar_init(s_empty + 8 * i, 8);  // the warps of a group
        }
        for (int i = 0; i < kLseSlots; ++i) {
            mbar_init(l_full + 8 * i, 1);
            mbar_init(l_empty + 8 * i, kSoftWarps);
        }
        mbar_init(fin, 1);
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
    int step = 1, xtiles = 2;
    const bool ascend = starts_ascend(p.query_start, p.R, p.T);
    if (MODE == kLse) {
        const int g = blockIdx.x * kThreads + threadIdx.x;
        if (!ascend && g == 0) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
        for (int r = g; ascend && r < p.R; r += gridDim.x * kThreads) {
            const Request x = request_of(p, r);
            if (x.m < 0 || x.m > x.n) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
            if (__ldg(p.lens + r) > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
        }
    }
    if (ascend) {
        step = split_tiles(p, sums, reinterpret_cast<int*>(base + SM::kMask));
        if (MODE == kSum) {
            // single tiles of keys while pairs would leave SMs without one
            total = flat_scan(p.R, [&](int r) { return item_count<MODE>(p, r, step, 2); }, sums);
            if (total < 2LL * p.sms) xtiles = 1;
        }
        __syncthreads();
        if (MODE == kLse || xtiles == 1)
            total = flat_scan(p.R, [&](int r) { return item_count<MODE>(p, r, step, xtiles); }, sums);
    }
    const int tr = kTile / p.G * p.G;
    auto item = [&](long long i) { return item_at<MODE>(p, sums, i, step, xtiles); };

    if (warp == kLoadWarp) {
        // ------------------------------------------------------- loads ----
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        uint32_t xc = 0, yc = 0;
        bool ok = true;
        // key tile j of the item's request to dst: 16-token blocks, each as kH
        // 64-column halves; returns the tile's mask of blocks in the cache
        auto load_keys = [&](const Item& it, uint32_t dst, uint32_t fb, int j, int tiles) {
            const int b0 = j * (kTile / kBlock), x = b0 + lane;
            bool have = lane < tiles * (kTile / kBlock) && x * kBlock < it.x.n;
            int blk = -1;
            if (have) {
                blk = __ldg(p.tables + (long long)it.r * p.mbps + x);
                have = blk >= 0 && blk < p.num_blocks;
                if (!have && MODE == kLse) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
            }
            const uint32_t msk = __ballot_sync(0xffffffffu, have);
            if (lane == 0) {
                if (MODE == kLse) sts32(mask0 + (yc % kMaskSlots) * 4, msk);
                mbar_arrive_expect_tx(fb, (uint32_t)__popc(msk) * kH * kBlock * 128u);
            }
            __syncwarp();
            if (have) {
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
        for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Item it = item(i);
            if (it.xt == 0 || it.y0 >= it.y1) continue;
            const uint32_t xs = xc & 1;
            if (!(ok = wait_warp(x_empty + 8 * xs, ((xc >> 1) & 1) ^ 1, p.wait_ns))) break;
            const uint32_t xd = sbase + SM::kX + xs * 2 * SM::kT;
            if (MODE == kLse)
                load_rows(it, xd, x_full + 8 * xs, it.row0, it.xt);
            else
                load_keys(it, xd, x_full + 8 * xs, it.row0 / kTile, it.xt);
            ++xc;
            for (int j = it.y0; j < it.y1; ++j, ++yc) {
                const uint32_t ys = yc % kYSlots;
                if (!(ok = wait_warp(y_empty + 8 * ys, ((yc / kYSlots) & 1) ^ 1, p.wait_ns))) break;
                if (p.withhold && yc == 0) continue;
                const uint32_t yd = sbase + SM::kY + ys * SM::kT;
                if (MODE == kLse)
                    load_keys(it, yd, y_full + 8 * ys, j, 1);
                else
                    load_rows(it, yd, y_full + 8 * ys, j * tr, 1);
            }
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
        for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Item it = item(i);
            if (it.xt == 0 || it.y0 >= it.y1) continue;
            if (!(ok = wait_warp(x_full + 8 * (xc & 1), (xc >> 1) & 1, p.wait_ns))) break;
            for (int j = it.y0; ok && j < it.y1; ++j, ++yc) {
                if (!(ok = wait_warp(y_full + 8 * (yc % kYSlots), (yc / kYSlots) & 1, p.wait_ns))) break;
                const uint32_t ya = sbase + SM::kY + (yc % kYSlots) * SM::kT;
                for (int t = 0; t < it.xt; ++t, ++sc) {
                    const uint32_t b = sc % kSBufs;
                    if (!(ok = wait_warp(s_empty + 8 * b, ((sc / kSBufs) & 1) ^ 1, p.wait_ns))) break;
                    tc::fence_after();
                    const uint32_t xa = sbase + SM::kX + ((xc & 1) * 2 + t) * SM::kT;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * kTile * 128 + (kk & 3) * 32;
                        tc::mma_ss_elect(tbase + b * kTile, tc::sdesc_sw128(xa + off, 16, 1024),
                                         tc::sdesc_sw128(ya + off, 16, 1024), id, kk > 0);
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
        if (MODE == kSum) {
            // -------------------------------- the rows' log-sum-exps ----
            uint32_t yc = 0;
            bool ok = true;
            for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
                const Item it = item(i);
                const int rows = it.x.m * p.G;
                for (int j = it.y0; j < it.y1; ++j, ++yc) {
                    const int nsp = ceil_div(seen_tiles(p, it.x, j >> 1), step);
                    float l[kTile / 32];
#pragma unroll
                    for (int u = 0; u < kTile / 32; ++u) {
                        const int c = u * 32 + lane, rho = j * tr + c;
                        float M = -INFINITY, sum = 0.f;
                        if (c < tr && rho < rows) {
                            const float* at = p.part + ((long long)(it.x.q0 + rho / p.G) * p.Hq + (long long)it.h * p.G + rho % p.G) * p.splits;
                            for (int s = 0; s < nsp; ++s) {
                                const float v = __ldcg(at + s);
                                const float n = fmaxf(M, v);
                                if (n != -INFINITY) sum = sum * exp2f(M - n) + exp2f(v - n);
                                M = n;
                            }
                        }
                        // a row without keys: every weight is 2^-inf
                        l[u] = sum > 0.f ? -(M + log2f(sum)) : -INFINITY;
                    }
                    const uint32_t ls = yc % kLseSlots;
                    if (!(ok = wait_warp(l_empty + 8 * ls, ((yc / kLseSlots) & 1) ^ 1, p.wait_ns))) break;
#pragma unroll
                    for (int u = 0; u < kTile / 32; ++u) lses[ls * kTile + u * 32 + lane] = l[u];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(l_full + 8 * ls);
                }
            }
            if (!ok && lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
        }
    } else {
        // ---------------------------------------------------- softmax ----
        const int group = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
        const int my = quad * 32 + lane;  // row of a tile, tensor-memory lane
        const uint32_t ts = tbase + ((uint32_t)(quad * 32) << 16) + 64u * half;
        const uint64_t sc2 = tc::f2(p.sl2, p.sl2);
        const bool pos_scale = p.sl2 > 0.f;
        const float off_value = pos_scale ? -INFINITY : INFINITY;  // a masked logit, before the scale
        uint32_t yc = 0, sc = 0, ic = 0;
        bool ok = true;
        for (long long i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Item it = item(i);
            if (it.xt == 0) continue;
            const int rows = it.x.m * p.G;
            // kLse: the last key this thread's row sees; kSum: the first row
            // that sees this thread's key
            const int tile = it.xt == 2 ? group ^ (int)(sc & 1) : 0;  // this group's S tiles of the item
            int bound;
            bool mine;
            if (MODE == kLse) {
                const int rho = it.row0 + tile * tr + my;
                mine = my < tr && rho < rows;
                bound = mine ? it.x.first + rho / p.G : 0x3FFFFFFF;
            } else {
                const int t = it.row0 + tile * kTile + my;
                mine = t < it.x.n;
                bound = mine ? max(0, t - it.x.first) * p.G : 0;
            }
            float m = -INFINITY;
            uint64_t acc[2] = {0ull, 0ull};
            for (int j = it.y0; ok && j < it.y1; ++j, ++yc) {
                if (MODE == kSum &&
                    !(ok = wait_warp(l_full + 8 * (yc % kLseSlots), (yc / kLseSlots) & 1, p.wait_ns)))
                    break;
                for (int t = 0; t < it.xt; ++t, ++sc) {
                    if ((int)(sc & 1) != group) continue;
                    const uint32_t b = sc % kSBufs;
                    if (!(ok = wait_warp(s_full + 8 * b, (sc / kSBufs) & 1, p.wait_ns))) break;
                    tc::fence_after();
                    uint32_t x[64];
                    tc::ld32(ts + b * kTile, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                    tc::ld32(ts + b * kTile + 32u, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
                    tc::wait_ld();
                    tc::fence_before();
                    __syncwarp();
                    if (MODE == kLse) {
                        const uint32_t msk = (lds32(mask0 + (yc % kMaskSlots) * 4) >> (4 * half)) & 0xFu;
                        if (lane == 0) mbar_arrive(s_empty + 8 * b);
                        const int key0 = j * kTile + 64 * half;
                        if (!__all_sync(0xffffffffu, msk == 0xFu && key0 + 63 <= bound)) {
#pragma unroll
                            for (int c = 0; c < 64; ++c)
                                if (!((msk >> (c >> 4)) & 1u) || key0 + c > bound) x[c] = __float_as_uint(off_value);
                        }
                        float e4[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) e4[c] = off_value;
                        if (pos_scale) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                e4[c & 3] = tc::max3(e4[c & 3], __uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1]));
                        } else {
#pragma unroll
                            for (int c = 0; c < 64; ++c) e4[c & 3] = fminf(e4[c & 3], __uint_as_float(x[c]));
                        }
                        const float ext = pos_scale ? fmaxf(fmaxf(e4[0], e4[1]), fmaxf(e4[2], e4[3]))
                                                    : fminf(fminf(e4[0], e4[1]), fminf(e4[2], e4[3]));
                        const float mn = fmaxf(m, ext * p.sl2);
                        const float u = mn == -INFINITY ? 0.f : mn;
                        const float al = ex2(m - u);
                        m = mn;
                        const uint64_t al2 = tc::f2(al, al), nu2 = tc::f2(-u, -u);
                        acc[0] = tc::fma2(acc[0], al2, 0ull);
                        acc[1] = tc::fma2(acc[1], al2, 0ull);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const uint64_t a = tc::fma2(tc::f2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, nu2);
                            acc[c & 1] = tc::add2(acc[c & 1], tc::f2(ex2(tc::f2_lo(a)), ex2(tc::f2_hi(a))));
                        }
                    } else {
                        if (lane == 0) mbar_arrive(s_empty + 8 * b);
                        const uint32_t la = sbase + SM::kLses + ((yc % kLseSlots) * kTile + 64 * half) * 4;
                        const int rho0 = j * tr + 64 * half, end = min(rows, (j + 1) * tr);
                        if (__all_sync(0xffffffffu, bound <= rho0) && rho0 + 64 <= end) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                uint32_t l0, l1, l2, l3;
                                lds128(la + 16 * c, l0, l1, l2, l3);
                                const uint64_t a0 = tc::fma2(tc::f2(__uint_as_float(x[4 * c]), __uint_as_float(x[4 * c + 1])), sc2,
                                                             tc::f2(__uint_as_float(l0), __uint_as_float(l1)));
                                const uint64_t a1 = tc::fma2(tc::f2(__uint_as_float(x[4 * c + 2]), __uint_as_float(x[4 * c + 3])), sc2,
                                                             tc::f2(__uint_as_float(l2), __uint_as_float(l3)));
                                acc[0] = tc::add2(acc[0], tc::f2(ex2(tc::f2_lo(a0)), ex2(tc::f2_hi(a0))));
                                acc[1] = tc::add2(acc[1], tc::f2(ex2(tc::f2_lo(a1)), ex2(tc::f2_hi(a1))));
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                const float l0 = __uint_as_float(lds32(la + 8 * c)), l1 = __uint_as_float(lds32(la + 8 * c + 4));
                                const int r0 = rho0 + 2 * c, r1 = r0 + 1;
                                const float w0 = r0 >= bound && r0 < end ? ex2(__fmaf_rn(__uint_as_float(x[2 * c]), p.sl2, l0)) : 0.f;
                                const float w1 = r1 >= bound && r1 < end ? ex2(__fmaf_rn(__uint_as_float(x[2 * c + 1]), p.sl2, l1)) : 0.f;
                                acc[c & 1] = tc::add2(acc[c & 1], tc::f2(w0, w1));
                            }
                        }
                    }
                }
                if (MODE == kSum) {
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(l_empty + 8 * (yc % kLseSlots));
                }
            }
            // the threads that share a row: two column halves, and for a
            // single tile the two groups
            const uint64_t a = tc::add2(acc[0], acc[1]);
            const float sum = tc::f2_lo(a) + tc::f2_hi(a);
            float2* comb = reinterpret_cast<float2*>(base + SM::kComb) + (ic & 1) * 4 * kTile;
            // a warp whose wait ran out still meets the others here, and all
            // of them leave together
            if (!ok && lane == 0) failed[ic & 1] = 1;
            comb[(half * 2 + group) * kTile + my] = make_float2(m, sum);
            asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
            if (failed[ic & 1]) {
                ok = false;
                break;
            }
            ++ic;
            if (half == 0 && mine && (it.xt == 2 || group == 0)) {
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
                        l > 0.f ? M + log2f(l) : -INFINITY;
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

// Places for partial log-sum-exps per row: enough splits that few row tiles
// still fill the GPU, fewer where the rows themselves are many.
int split_places(const mi_dims& D, int32_t total_q) {
    const long long rows = (long long)total_q * D.Hq;
    return rows <= (1LL << 20) ? 32 : rows <= (1LL << 23) ? 8 : 2;
}

size_t window_bytes(const mi_dims& D, int32_t total_q) {
    return ((size_t)total_q * D.Hq * split_places(D, total_q) * 4 + 255) / 256 * 256 + 256;
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
    p.part = static_cast<float*>(workspace);
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
    const bool ok = HD == 128 ? launch_window<128, kLse>(tq, tk, p, st) && launch_window<128, kSum>(tq, tk, p, st)
                              : launch_window<64, kLse>(tq, tk, p, st) && launch_window<64, kSum>(tq, tk, p, st);
    return ok ? MI_OK : MI_ERR_CUDA;
}
