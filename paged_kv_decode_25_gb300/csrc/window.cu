// mi_paged_prefill_scores: the attention weight every cached token receives
// from many query tokens at once (the last tokens of a prompt, or all of it).
//
//   score[r][h][t] (+)= sum over query tokens i of request r with t <= pos_i
//                       and the G query heads j of h of 2^(x_ijt - lse_ij)
//
// A weight needs its row's log-sum-exp over all keys, so the logits x are
// computed twice: the first launch reduces them over the keys of each row, the
// second over the rows of each key. (Kept
// in memory they would be 4 bytes a pair each way, 0.5 GB for 16 windows of 64
// tokens over 85,000 keys; the second product costs a tenth of that time.) V is
// never read.
//
// The two are one pipeline on the fifth-generation tensor cores: an item keeps
// X in shared memory and streams Y past it, S = A . B^T in tiles of 128 x 256:
//   * kLse: X = up to 256 (query token, head) rows of a request (A, 128 a
//     tile), Y = its keys (B, 256 a stage); a row's keys may be split over
//     several items (partial log-sum-exps);
//   * kSum: X = up to 256 keys (A, 128 a tile), Y = query rows (B, 256 a
//     stage), from the first that sees a key; a small launch before it merges
//     the rows' partial log-sum-exps, which it reads once per 256 keys;
//   * kWindow, where no request has more than 256 rows: X = those rows (B), Y =
//     keys (A, 128 a stage), so that a key is finished with its stage and K
//     streams past resident rows (with K resident the rows would be streamed
//     again for every 256 keys, twice the traffic).
// A thread owns a row of S (a tensor-memory lane) and a quarter of its columns,
// so both reductions are private to a thread until the item's end (kWindow: the
// stage's).
//   warps 0-15   softmax, all on the same S tile while the tensor cores fill the
//                other: warp w takes lanes 32 (w mod 4) .. + 31 and columns
//                64 (w / 4) .. + 63 (with a tile per eight warps, each half
//                waited for its own next tile a third of the time)
//   warp 16      issues the MMAs and owns the tensor memory (two S tiles)
//   warp 17      picks the items, streams X and Y
//   warp 18      the query rows' log-sum-exps (kSum, kWindow)
// Why 256 columns: an MMA of 128 x 128 x 16 takes 63 clocks to issue whatever
// its size, and a tile's waits and commits another 360, so tiles of 128
// columns ran at 868 clocks against 512 of tensor core; one of 256 takes 1,038
// against 1,024 (measured apart from the softmax).
//
// Measured (head_dim 128, 32 heads over 8): 16 windows of 32 to 64 tokens over
// 77,600 keys 48 + 49 us, each with two or three items a block that cost 7,000
// clocks to start (X has one place) on top of 30 tiles; two whole prompts of
// 5,000 tokens 190 + 10 + 164 us, 565 TFLOP/s of the products it cannot do
// without. No unit bounds the latter: a tile of 32,768 logits takes 1,300 to
// 1,500 clocks, of which its exponentials are 1,024, the issue slots are used
// for 48 to 53 % and the tensor cores for 47 to 54 %; what is lost lies in the
// hand-over from tile to tile and in the items' starts.
#include <cmath>

#include "batch.cuh"
#include "tc.cuh"
#include "window.cuh"

namespace mi {
namespace {

using namespace window;

constexpr int kSoftWarps = 16, kQuarters = 4, kMmaWarp = 16, kLoadWarp = 17, kLseWarp = 18;
constexpr int kThreads = 19 * 32;
constexpr int kMaskSlots = 16, kLseSlots = 4, kItemSlots = 4;
constexpr uint32_t kCols = 512;
constexpr int kMergeThreads = 256;

template <int HD, int MODE>
struct WinSmem {
    static constexpr int kH = HD / 64;
    // Both layouts with 128-byte swizzle. Query rows: [kH][256 rows][128 B].
    // Keys: [groups of 8 rows][kH][8 rows][128 B], so that one copy brings a
    // block whole (with the halves apart it takes kH copies, 72 clocks each to
    // issue: 1,150 for 128 keys, more than their products).
    static constexpr int kRowBytes = kH * kRows * 128, kKeyBytes = kH * kKeys * 128;
    static constexpr int kXBytes = kRowBytes;             // 256 rows or 256 keys
    static constexpr int kYBytes = MODE == kWindow ? kKeyBytes : kRowBytes;
    static constexpr int kXSlots = 65536 / kXBytes, kYSlots = 131072 / kYBytes;
    static constexpr int kX = 0;
    static constexpr int kY = 65536;
    static constexpr int kLses = kY + 131072;             // [kLseSlots][256] fp32
    static constexpr int kComb = kLses + kLseSlots * kRows * 4;  // [2][2 tiles][kQuarters][128] float2
    static constexpr int kItems = kComb + 4 * kQuarters * kKeys * 8;
    static constexpr int kSums = kItems + kItemSlots * 64;
    static constexpr int kMask = kSums + flat_words(kThreads) * 8;
    static constexpr int kBar = (kMask + kMaskSlots * 4 + 7) / 8 * 8;
    static constexpr int kNBar = 2 * kXSlots + 2 * kYSlots + 4 + 2 * kLseSlots + 2 * kItemSlots + 1 + 4;
    static constexpr int kTmem = kBar + kNBar * 8;        // the tensor-memory base, then two words: a wait ran out
    static constexpr int kTotal = kTmem + 16 + 1024;      // slack to align the base to 1024 B
};

// One work item: X of xt tiles of 128 (0: the list is over), Y stages y0 .. y1-1.
struct __align__(16) Item {
    int r, h, xt, y0, y1, row0, slot, pad;  // row0: the first query row (kLse) or key (kSum) of X
    Request x;
};
static_assert(sizeof(Item) <= 64, "an item's place in shared memory");

// Rows row, row + 32, ..: all of a part's loads at once.
template <int N>
__device__ __forceinline__ void merge_rows(const RowParts& v, int row, float (&out)[N]) {
    float M[N], sum[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        M[u] = -INFINITY;
        sum[u] = 0.f;
    }
#pragma unroll 2
    for (int s = 0; s < v.n; ++s) {
        float l[N];
#pragma unroll
        for (int u = 0; u < N; ++u) l[u] = __ldcg(v.at + s * kRows + row + 32 * u);
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const float top = fmaxf(M[u], l[u]);
            if (top > -INFINITY) {
                sum[u] = sum[u] * exp2f(M[u] - top) + exp2f(l[u] - top);
                M[u] = top;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) out[u] = sum[u] == 0.f ? -INFINITY : -(M[u] + log2f(sum[u]));
}

// kSum's items: 128 xkeys keys of a head.
__device__ __forceinline__ long long sum_items(const WindowParams& p, int r, int xkeys) {
    const Request x = request_of(p, r);
    return x.m < 0 ? 0 : (long long)p.Hkv * ceil_div(x.n, xkeys * kKeys);
}
__device__ __forceinline__ Item sum_item(const WindowParams& p, const long long* sums, long long i, int xkeys) {
    Item it;
    long long first;
    it.r = flat_find(p.R, [&](int r) { return sum_items(p, r, xkeys); }, sums, i, first);
    it.x = request_of(p, it.r);
    const int o = (int)(i - first), rp = p.tokens * p.G;
    it.h = o % p.Hkv;
    it.slot = 0;
    it.row0 = o / p.Hkv * xkeys * kKeys;
    it.xt = min(xkeys, ceil_div(it.x.n - it.row0, kKeys));
    it.y0 = max(0, it.row0 - it.x.first) * p.G / rp;  // rows before it see none of the keys
    it.y1 = max(it.y0, ceil_div(it.x.m * p.G, rp));
    return it;
}
// A share's units in order, from the one at cost `pos` on.
template <int MODE>
struct Units {
    Item it;
    Cost c;
    long long first;  // the cost before the request
    int rb;

    __device__ __forceinline__ void row_block(const WindowParams& p, int h) {
        it.h = h;
        if (MODE == kLse) {
            c = lse_cost(p, it.x, rb, h, first);
            it.row0 = rb * p.tokens * p.G;
            it.xt = it.x.m * p.G - it.row0 > kKeys ? 2 : 1;
        } else {
            const int w = kUnitTiles + ceil_div(it.x.n, kKeys);
            c.at = first + (long long)h * w;
            c.end = c.at + w;
            c.start = kUnitTiles;
            c.per = 1;
            c.stages = w - kUnitTiles;
            it.row0 = it.slot = 0;
            it.xt = 1;
        }
    }
    __device__ __forceinline__ void seek(const WindowParams& p, const long long* sums, long long pos) {
        it.r = flat_find(p.R, [&](int r) { return request_cost<MODE>(p, r); }, sums, pos, first);
        it.x = request_of(p, it.r);
        rb = 0;
        if (MODE == kLse) {
            int hi = row_blocks(p, it.x);
            while (hi - rb > 1) {
                const int mid = (rb + hi) >> 1;
                if (first + p.Hkv * cost_before(p, it.x, mid) <= pos) rb = mid;
                else hi = mid;
            }
        }
        row_block(p, 0);
        const int h = small_quotient(pos - c.at, c.end - c.at);
        if (h > 0) row_block(p, h);
    }
    // The unit's stages up to the share's end.
    __device__ __forceinline__ void stages(const WindowParams& p, long long pos, long long stop) {
        it.y0 = c.reaches(pos);
        it.y1 = c.reaches(min(stop, c.end));
        if (MODE == kLse) it.slot = lse_unit(p, it.x, rb, it.h) + (int)blockIdx.x;
    }
    // The next unit, which begins where this one ends (before the share does).
    __device__ __forceinline__ void advance(const WindowParams& p, const long long* sums) {
        const long long w = c.end - c.at;
        if (it.h + 1 < p.Hkv) {
            ++it.h;
            c.at = c.end;
            c.end += w;
        } else if (MODE == kLse && rb + 1 < row_blocks(p, it.x)) {
            ++rb;
            row_block(p, 0);
        } else {
            seek(p, sums, c.end);
        }
    }
};

// Whether phase `parity` of the barrier has completed, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// f(x, q) for the two chunks of 32 columns of a warp's quarter at ts, the second
// loaded under the arithmetic of the first; done() once both are in registers.
template <typename F, typename D>
__device__ __forceinline__ void sweep(uint32_t ts, F f, D done) {
    uint32_t xa[32], xb[32];
    tc::ld32(ts, xa);
    tc::wait_ld();
    tc::ld32(ts + 32u, xb);
    f(xa, 0);
    tc::wait_ld();
    done();
    f(xb, 1);
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n > 0 ? (1u << n) - 1u : 0u; }
// Columns of a chunk without their bit in `keep` take the value `off`.
__device__ __forceinline__ void cut(uint32_t (&x)[32], uint32_t keep, float off) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (!(keep & (1u << c))) x[c] = __float_as_uint(off);
}
// kLse: bit i of `have`: the quarter's columns 16 i .. + 15 hold keys; the row
// sees columns below `hi`. The columns of chunk q that count.
__device__ __forceinline__ uint32_t seen_columns(uint32_t have, int hi, int q) {
    const uint32_t two = have >> (2 * q);
    return low_bits(hi - 32 * q) & ((two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u));
}
template <bool HIGHEST>
__device__ __forceinline__ float chunk_top(const uint32_t (&x)[32]) {
    auto pick = [](float a, float b) { return HIGHEST ? fmaxf(a, b) : fminf(a, b); };
    float e4[4];
#pragma unroll
    for (int c = 0; c < 32; ++c)
        e4[c & 3] = c < 4 ? __uint_as_float(x[c]) : pick(e4[c & 3], __uint_as_float(x[c]));
    return pick(pick(e4[0], e4[1]), pick(e4[2], e4[3]));
}

// acc += 2^(x sc2 + b) over a chunk.
__device__ __forceinline__ void add_chunk(const uint32_t (&x)[32], uint64_t sc2, uint64_t b, uint64_t (&acc)[4]) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const uint64_t a = tc::fma2(tc::f2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, b);
        acc[c & 3] = tc::add2(acc[c & 3], tc::f2(ex2(tc::f2_lo(a)), ex2(tc::f2_hi(a))));
    }
}
// As above with b the 32 values at shared address la.
__device__ __forceinline__ void add_chunk_rows(const uint32_t (&x)[32], uint64_t sc2, uint32_t la, uint64_t (&acc)[4]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t l0, l1, l2, l3;
        lds128(la + 16 * c, l0, l1, l2, l3);
        const uint64_t a0 = tc::fma2(tc::f2(__uint_as_float(x[4 * c]), __uint_as_float(x[4 * c + 1])), sc2,
                                     tc::f2(__uint_as_float(l0), __uint_as_float(l1)));
        const uint64_t a1 = tc::fma2(tc::f2(__uint_as_float(x[4 * c + 2]), __uint_as_float(x[4 * c + 3])), sc2,
                                     tc::f2(__uint_as_float(l2), __uint_as_float(l3)));
        acc[(2 * c) & 3] = tc::add2(acc[(2 * c) & 3], tc::f2(ex2(tc::f2_lo(a0)), ex2(tc::f2_hi(a0))));
        acc[(2 * c + 1) & 3] = tc::add2(acc[(2 * c + 1) & 3], tc::f2(ex2(tc::f2_lo(a1)), ex2(tc::f2_hi(a1))));
    }
}
__device__ __forceinline__ float total_of(const uint64_t (&acc)[4]) {
    const uint64_t a = tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3]));
    return tc::f2_lo(a) + tc::f2_hi(a);
}

// The sweeps that few tiles need (a mask, a first maximum) are functions of
// their own: inlined, the mask's selects and their registers slowed the plain
// sweep by a fifth.
__device__ __noinline__ float masked_top(uint32_t ts, uint32_t have, int hi, float sl2) {
    const float off = sl2 > 0.f ? -INFINITY : INFINITY;
    float best = off;
    sweep(ts, [&](uint32_t (&x)[32], int q) {
        cut(x, seen_columns(have, hi, q), off);
        best = sl2 > 0.f ? fmaxf(best, chunk_top<true>(x)) : fminf(best, chunk_top<false>(x));
    }, [] {});
    return best * sl2;
}
__device__ __noinline__ float masked_keys(uint32_t ts, uint32_t have, int hi, float sl2, float nu) {
    const float off = sl2 > 0.f ? -INFINITY : INFINITY;
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
    sweep(ts, [&](uint32_t (&x)[32], int q) {
        cut(x, seen_columns(have, hi, q), off);
        add_chunk(x, tc::f2(sl2, sl2), tc::f2(nu, nu), acc);
    }, [] {});
    return total_of(acc);
}
// A row's first tile: {m, the sum relative to 2^m}. A row without an m takes the
// largest logit of the first 32 columns, or of the others where those hold none
// of it.
__device__ __noinline__ float2 first_keys(uint32_t ts, uint32_t have, int hi, float sl2, float m) {
    const float off = sl2 > 0.f ? -INFINITY : INFINITY;
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
    sweep(ts, [&](uint32_t (&x)[32], int q) {
        cut(x, seen_columns(have, hi, q), off);
        if (m == -INFINITY) m = (sl2 > 0.f ? chunk_top<true>(x) : chunk_top<false>(x)) * sl2;
        const float nu = m == -INFINITY ? 0.f : -m;
        add_chunk(x, tc::f2(sl2, sl2), tc::f2(nu, nu), acc);
    }, [] {});
    return make_float2(m, total_of(acc));
}
// Columns from `first` on see the thread's key, `cols` hold rows.
__device__ __noinline__ float masked_rows(uint32_t ts, uint32_t la, int first, int cols, float sl2) {
    const float off = sl2 > 0.f ? -INFINITY : INFINITY;
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
    sweep(ts, [&](uint32_t (&x)[32], int q) {
        if (32 * q >= cols) return;
        cut(x, low_bits(cols - 32 * q) & ~low_bits(first - 32 * q), off);
        add_chunk_rows(x, tc::f2(sl2, sl2), la + 128 * q, acc);
    }, [] {});
    return total_of(acc);
}

template <int HD, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const WindowParams p) {
    using SM = WinSmem<HD, MODE>;
    constexpr int kH = SM::kH, kXSlots = SM::kXSlots, kYSlots = SM::kYSlots;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
    unsigned char* base = smem_raw + (sbase - raw);
    long long* sums = reinterpret_cast<long long*>(base + SM::kSums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sbase + SM::kBar;
    const uint32_t x_full = bar, x_empty = x_full + 8 * kXSlots, y_full = x_empty + 8 * kXSlots;
    const uint32_t y_empty = y_full + 8 * kYSlots, s_full = y_empty + 8 * kYSlots, s_empty = s_full + 16;
    const uint32_t l_full = s_empty + 16, l_empty = l_full + 8 * kLseSlots;
    const uint32_t i_full = l_empty + 8 * kLseSlots, i_empty = i_full + 8 * kItemSlots, fin = i_empty + 8 * kItemSlots;
    const uint32_t c_full = fin + 8;  // kWindow: [4 places] the other quarters' sums
    volatile int* failed = reinterpret_cast<volatile int*>(base + SM::kTmem + 4);
    const uint32_t mask0 = sbase + SM::kMask;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kXSlots; ++i) {
            mbar_init(x_full + 8 * i, 1);
            mbar_init(x_empty + 8 * i, 1);
        }
        for (int i = 0; i < kYSlots; ++i) {
            mbar_init(y_full + 8 * i, 1);
            mbar_init(y_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 2);   // the MMAs' commit, and the issuing warp (for what it has seen)
            mbar_init(s_empty + 8 * i, kSoftWarps);
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
        for (int i = 0; i < 4; ++i) mbar_init(c_full + 8 * i, kSoftWarps - 4);
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
    // ---------------------------------------------------------- the plan --
    // the launches after kLse plan while the one before them ends: the requests
    // were there before the first
    if (MODE == kLse) {
        pdl_wait();
        pdl_trigger();
    }
    long long total = 0, pos = 0, stop = 0, share = 0;  // share: kLse's
    int xkeys = 2;
    bool ascend = true;
    if (MODE == kLse) {
        ascend = starts_ascend(p.query_start, p.R, p.T);
        const int g = blockIdx.x * kThreads + threadIdx.x;
        if (!ascend && g == 0) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
        for (int r = g; ascend && r < p.R; r += gridDim.x * kThreads) {
            const Request x = request_of(p, r);
            if (x.m < 0 || x.m > x.n) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
            if (__ldg(p.lens + r) > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
        }
        if (!ascend && g == 0) p.begin[p.R] = 0;
    }
    if (ascend && MODE == kSum) {
        total = flat_scan(p.R, [&](int r) { return sum_items(p, r, xkeys); }, sums);
        if (total < 2LL * gridDim.x) {
            // 128 keys an item while 256 would leave SMs with few
            xkeys = 1;
            __syncthreads();
            total = flat_scan(p.R, [&](int r) { return sum_items(p, r, xkeys); }, sums);
        }
    } else if (ascend) {
        auto cost = [&](int r) { return request_cost<MODE>(p, r); };
        total = flat_scan(p.R, cost, sums);
        const long long mine = even_share(total, gridDim.x, MODE);
        pos = blockIdx.x * mine;
        stop = min(pos + mine, total);
        if (MODE == kLse) {
            for (int r = blockIdx.x + gridDim.x * threadIdx.x; r < p.R; r += gridDim.x * kThreads)
                p.begin[r] = flat_before(p.R, cost, sums, r);
            if (blockIdx.x == 0 && threadIdx.x == 0) p.begin[p.R] = mine;
        }
    }
    if (MODE != kLse) {
        pdl_wait();
        pdl_trigger();
        share = __ldcg(p.begin + p.R);
        if (share == 0) total = stop = 0;
    }
    const int rp = p.tokens * p.G;
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
        // the lane's block of `tiles` key tiles from tile j on (-1: none; -2: not in the cache)
        auto entry = [&](const Item& it, int j, int tiles) -> int {
            const int x = j * (kKeys / kBlock) + lane;
            if (lane >= tiles * (kKeys / kBlock) || x * kBlock >= it.x.n) return -1;
            const int blk = __ldg(p.tables + (long long)it.r * p.mbps + x);
            return blk >= 0 && blk < p.num_blocks ? blk : -2;
        };
        // those blocks to dst; kLse posts the stage's mask of blocks in the cache
        auto load_keys = [&](const Item& it, uint32_t dst, uint32_t fb, int blk) {
            if (MODE == kLse && blk == -2) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
            const uint32_t msk = __ballot_sync(0xffffffffu, blk >= 0);
            if (lane == 0) {
                if (MODE == kLse) sts32(mask0 + (yc % kMaskSlots) * 4, msk);
                mbar_arrive_expect_tx(fb, (uint32_t)__popc(msk) * kH * kBlock * 128u);
            }
            __syncwarp();
            if (blk >= 0)
                tma_load_4d(dst + lane * kH * kBlock * 128, &tmk, fb, 0, 0, 0, (blk * p.Hkv + it.h) * (kBlock / 8), policy);
        };
        // the block of query rows from row0 on
        auto load_rows = [&](const Item& it, uint32_t dst, uint32_t fb, int row0) {
            if (lane == 0) {
                mbar_arrive_expect_tx(fb, (uint32_t)(kH * rp) * 128u);
                for (int hh = 0; hh < kH; ++hh)
                    tma_load_4d(dst + hh * kRows * 128, &tmq, fb, 0, hh, it.h * p.G, it.x.q0 + row0 / p.G, policy);
            }
            __syncwarp();
        };
        // kSum's items (of very different lengths, the longest first) are taken
        // from a counter, each when the last stage of the one before is out:
        // taken earlier, long ones wait behind others (a third of the time)
        Units<MODE> units;
        units.c.end = -1;  // none yet
        auto pick = [&]() -> Item {
            Item it;
            it.xt = 0;
            if (MODE == kSum) {
                unsigned int i = 0;
                if (lane == 0) i = atomicAdd(p.next, 1u);
                i = __shfl_sync(0xffffffffu, i, 0);
                if (i < total) it = sum_item(p, sums, i, xkeys);
            } else {
                while (pos < stop) {
                    if (units.c.end < 0) units.seek(p, sums, pos);
                    else units.advance(p, sums);
                    units.stages(p, pos, stop);
                    pos = units.c.end;
                    if (units.it.y0 < units.it.y1) {
                        it = units.it;
                        break;
                    }
                }
            }
            return it;
        };
        uint32_t ic = 0;
        for (;;) {
            const Item it = pick();
            const uint32_t sl = ic % kItemSlots;
            if (!(ok = wait_warp(i_empty + 8 * sl, ((ic / kItemSlots) & 1) ^ 1, p.wait_ns))) break;
            if (lane == 0) {
                *reinterpret_cast<Item*>(base + SM::kItems + sl * 64) = it;
                mbar_arrive(i_full + 8 * sl);
            }
            __syncwarp();
            ++ic;
            if (it.xt == 0) break;
            if (it.y0 >= it.y1) continue;
            // X goes out first where its place is free, and at the latest
            // before a wait for Y's ring: an item's first Y stages may land
            // while the last item still holds X
            const uint32_t xs = xc % kXSlots, xd = sbase + SM::kX + xs * SM::kXBytes;
            const int xblk = MODE == kSum ? entry(it, it.row0 / kKeys, it.xt) : 0;
            bool have_x = false;
            auto load_x = [&]() -> bool {
                have_x = true;
                if (!wait_warp(x_empty + 8 * xs, ((xc / kXSlots) & 1) ^ 1, p.wait_ns)) return false;
                if (MODE == kSum)
                    load_keys(it, xd, x_full + 8 * xs, xblk);
                else
                    load_rows(it, xd, x_full + 8 * xs, it.row0);
                ++xc;
                return true;
            };
            // table entries are read a stage ahead of their use
            constexpr int yt = MODE == kLse ? 2 : 1;  // key tiles of a stage
            int blk = MODE == kSum ? 0 : entry(it, it.y0 * yt, yt);
            if (__all_sync(0xffffffffu, mbar_test_wait(x_empty + 8 * xs, ((xc / kXSlots) & 1) ^ 1)) && !(ok = load_x())) break;
            for (int j = it.y0; j < it.y1; ++j, ++yc) {
                const int now = blk;
                if (MODE != kSum && j + 1 < it.y1) blk = entry(it, (j + 1) * yt, yt);
                const uint32_t ys = yc % kYSlots, yp = ((yc / kYSlots) & 1) ^ 1;
                if (!have_x && !__all_sync(0xffffffffu, mbar_test_wait(y_empty + 8 * ys, yp)) && !(ok = load_x())) break;
                if (!(ok = wait_warp(y_empty + 8 * ys, yp, p.wait_ns))) break;
                if (p.withhold && yc == 0) continue;
                const uint32_t yd = sbase + SM::kY + ys * SM::kYBytes;
                if (MODE == kSum)
                    load_rows(it, yd, y_full + 8 * ys, j * rp);
                else
                    load_keys(it, yd, y_full + 8 * ys, now);
            }
            if (ok && !have_x) ok = load_x();
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
            // copies issued land before the block's shared memory goes away
            for (uint32_t s = 0; s < kXSlots; ++s)
                if (xc > s) (void)wait_warp(x_full + 8 * s, ((xc - 1 - s) / kXSlots) & 1, drain_limit(p.wait_ns));
            for (uint32_t s = p.withhold ? 1 : 0; s < kYSlots; ++s)
                if (yc > s) (void)wait_warp(y_full + 8 * s, ((yc - 1 - s) / kYSlots) & 1, drain_limit(p.wait_ns));
        }
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------- MMA issuer ----
        const uint32_t id = tc::idesc_bf16(kKeys, MODE == kWindow ? kKeys * p.xt : kRows, false);
        uint32_t xc = 0, yc = 0, sc = 0;
        bool ok = true;
        for (uint32_t ic = 0; ok; ++ic) {
            Item it;
            if (!(ok = take(ic, it)) || it.xt == 0) break;
            if (it.y0 >= it.y1) continue;
            const uint32_t xs = xc % kXSlots, xa = sbase + SM::kX + xs * SM::kXBytes;
            if (!(ok = wait_warp(x_full + 8 * xs, (xc / kXSlots) & 1, p.wait_ns))) break;
            for (int j = it.y0; ok && j < it.y1; ++j, ++yc) {
                const uint32_t ys = yc % kYSlots, ya = sbase + SM::kY + ys * SM::kYBytes;
                if (!(ok = wait_warp(y_full + 8 * ys, (yc / kYSlots) & 1, p.wait_ns))) break;
                for (int t = 0; t < it.xt; ++t, ++sc) {
                    const uint32_t b = sc & 1;
                    if (!(ok = wait_warp(s_empty + 8 * b, ((sc >> 1) & 1) ^ 1, p.wait_ns))) break;
                    tc::fence_after();
                    // query rows: 8-row groups 1024 B apart, halves 256 rows;
                    // keys: groups kH * 1024 B apart, halves 1024 B
                    const uint32_t ra = MODE == kSum ? ya : MODE == kLse ? xa + t * kKeys * 128 : xa;
                    const uint32_t ka = MODE == kSum ? xa + t * SM::kKeyBytes : ya;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t in = (kk & 3) * 32;  // 16 bf16 of a 128-byte row
                        const uint64_t rd = tc::sdesc_sw128(ra + (kk >> 2) * kRows * 128 + in, 16, 1024);
                        const uint64_t kd = tc::sdesc_sw128(ka + (kk >> 2) * 1024 + in, 16, kH * 1024);
                        tc::mma_ss_elect(tbase + b * kRows, MODE == kLse ? rd : kd, MODE == kLse ? kd : rd, id, kk > 0);
                    }
                    tc::commit_elect(s_full + 8 * b);
                    if (lane == 0) mbar_arrive(s_full + 8 * b);
                    __syncwarp();
                }
                if (ok) tc::commit_elect(y_empty + 8 * ys);
            }
            if (ok) tc::commit_elect(x_empty + 8 * xs);
            ++xc;
        }
        if (!ok && lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
        // every MMA issued has finished before tensor memory is released
        tc::commit_elect(fin);
        (void)wait_warp(fin, 0, drain_limit(p.wait_ns));
    } else if (warp == kLseWarp) {
        if (MODE != kLse) {
            // -------------------------------- the rows' log-sum-exps ----
            // Zero past a block's rows. kSum: a slot per Y stage, copied without
            // a wait, so the ring is filled ahead; kWindow: one per item, put
            // together here (a launch for it took 8 us of a step, and a row is
            // wanted a few times only).
            uint32_t lc = 0;
            bool ok = true;
            for (uint32_t ic = 0; ok; ++ic) {
                Item it;
                if (!(ok = take(ic, it)) || it.xt == 0) break;
                const int rows = it.x.m * p.G;
                if (MODE == kWindow) {
                    const uint32_t ls = lc++ % kLseSlots;
                    if (!(ok = wait_warp(l_empty + 8 * ls, (((lc - 1) / kLseSlots) & 1) ^ 1, p.wait_ns))) break;
                    float v[kRows / 32];
                    merge_rows(row_parts(p, it.x, it.r, 0, it.h, share), lane, v);
#pragma unroll
                    for (int u = 0; u < kRows / 32; ++u) {
                        const int c = u * 32 + lane;
                        sts32(sbase + SM::kLses + (ls * kRows + c) * 4, __float_as_uint(c < rows ? v[u] : 0.f));
                    }
                    mbar_arrive(l_full + 8 * ls);
                    continue;
                }
                const float* at = p.nlse + ((long long)it.h * p.T + it.x.q0) * p.G;
                for (int j = it.y0; j < it.y1; ++j, ++lc) {
                    const uint32_t ls = lc % kLseSlots;
                    if (!(ok = wait_warp(l_empty + 8 * ls, ((lc / kLseSlots) & 1) ^ 1, p.wait_ns))) break;
#pragma unroll
                    for (int u = 0; u < kRows / 32; ++u) {
                        const int c = u * 32 + lane, rho = j * rp + c;
                        const bool in = c < rp && rho < rows;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                         sbase + SM::kLses + (ls * kRows + c) * 4),
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
        const int quarter = warp >> 2, quad = warp & 3;
        const int my = quad * 32 + lane;  // row of a tile, tensor-memory lane
        const int col0 = quarter * 64;    // of this warp's columns
        const uint32_t ts0 = tbase + ((uint32_t)(quad * 32) << 16) + (uint32_t)col0;
        const uint64_t sc2 = tc::f2(p.sl2, p.sl2);
        uint32_t yc = 0, sc = 0;
        bool ok = true;
        auto give_back = [&](uint32_t b) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_empty + 8 * b);
        };
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
            // per tile: kLse: the last key this thread's row sees; kSum: the
            // first row that sees this thread's key
            int bound[2] = {0, 0};
            bool mine[2] = {false, false};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (MODE == kLse) {
                    const int rho = it.row0 + t * kKeys + my;
                    mine[t] = t < it.xt && t * kKeys + my < rp && rho < rows;
                    bound[t] = mine[t] ? it.x.first + rho / p.G : 0x3FFFFFFF;
                } else if (MODE == kSum) {
                    const int key = it.row0 + t * kKeys + my;
                    mine[t] = t < it.xt && key < it.x.n;
                    bound[t] = mine[t] ? max(0, key - it.x.first) * p.G : 0;
                }
            }
            float m[2] = {-INFINITY, -INFINITY};  // kLse: the sums are relative to 2^m
            float sum[2] = {0.f, 0.f};
            if (MODE == kWindow)
                ok = ok && wait_warp(l_full + 8 * (ic % kLseSlots), (ic / kLseSlots) & 1, p.wait_ns);
            for (int j = it.y0; ok && j < it.y1; ++j, ++yc) {
                if (MODE == kSum &&
                    !(ok = wait_warp(l_full + 8 * (yc % kLseSlots), (yc / kLseSlots) & 1, p.wait_ns)))
                    break;
                const int key = j * kKeys + my;  // kWindow: this thread's key of the stage, and its block
                int blk = -1;
                if (MODE == kWindow && quarter == 0 && key < it.x.n)
                    blk = __ldg(p.tables + (long long)it.r * p.mbps + key / kBlock);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= it.xt || !ok) continue;
                    const uint32_t b = sc & 1;
                    if (!(ok = wait_warp(s_full + 8 * b, (sc >> 1) & 1, p.wait_ns))) continue;
                    tc::fence_after();
                    const uint32_t ts = ts0 + b * kRows;
                    float got = 0.f;  // the tile's sum
                    if (MODE == kLse) {
                        const int key0 = j * 2 * kKeys + col0;
                        const uint32_t msk = (lds32(mask0 + (yc % kMaskSlots) * 4) >> (4 * quarter)) & 0xFu;
                        const bool part = __any_sync(0xffffffffu, msk != 0xFu || key0 + 63 > bound[t]);
                        const int hi = bound[t] - key0 + 1;
                        // The sum is relative to m, a large logit of the row's
                        // first tile: fp32 holds it however far others lie
                        // below, and above until it nears overflow. Only then
                        // is a maximum taken and the sum moved to it.
                        if (__any_sync(0xffffffffu, m[t] == -INFINITY)) {
                            const float2 v = first_keys(ts, msk, hi, p.sl2, m[t]);
                            m[t] = v.x;
                            got = v.y;
                        } else if (part) {
                            got = masked_keys(ts, msk, hi, p.sl2, -m[t]);
                        } else {
                            const uint64_t nu2 = tc::f2(-m[t], -m[t]);
                            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
                            sweep(ts, [&](uint32_t (&x)[32], int) { add_chunk(x, sc2, nu2, acc); }, [] {});
                            got = total_of(acc);
                        }
                        if (__any_sync(0xffffffffu, sum[t] + got > 0x1p100f)) {
                            const float best = masked_top(ts, msk, hi, p.sl2);
                            if (best > m[t]) {
                                sum[t] *= ex2(m[t] - best);
                                m[t] = best;
                            }
                            got = masked_keys(ts, msk, hi, p.sl2, m[t] == -INFINITY ? 0.f : -m[t]);
                        }
                        sum[t] += got;
                        give_back(b);
                    } else {
                        // the Y rows of kSum, the X rows of kWindow: of this
                        // warp's columns those from `first` on see the thread's
                        // key, and `cols` hold rows
                        const int row0 = (MODE == kSum ? j * rp : 0) + col0;
                        const int cols = min(min(rp - col0, 64), rows - row0);
                        const int first = (MODE == kSum ? bound[t] : max(key - it.x.first, 0) * p.G) - row0;
                        const bool part = __any_sync(0xffffffffu, first > 0) || cols < 64;
                        const uint32_t la = sbase + SM::kLses + (((MODE == kSum ? yc : ic) % kLseSlots) * kRows + col0) * 4;
                        if (cols <= 0) {
                            give_back(b);
                        } else if (part) {
                            got = masked_rows(ts, la, first, cols, p.sl2);
                            give_back(b);
                        } else {
                            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
                            sweep(ts, [&](uint32_t (&x)[32], int q) { add_chunk_rows(x, sc2, la + 128 * q, acc); },
                                  [&] { give_back(b); });  // as soon as it is in registers
                            got = total_of(acc);
                        }
                        if (MODE == kSum) sum[t] += got;
                    }
                    if (MODE == kWindow) {
                        // the other quarters hand their sums to the first one
                        // through one of four places: they come to a place
                        // again four S tiles on, and the tile before the last
                        // of these is given back by the first quarter only
                        // once it is done with this place
                        const int place = (int)(sc & 3);
                        float* comb = reinterpret_cast<float*>(base + SM::kComb) + place * 3 * kKeys;
                        float w = got;
                        if (quarter > 0) {
                            comb[(quarter - 1) * kKeys + my] = w;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(c_full + 8 * place);
                        } else {
                            if (!(ok = wait_warp(c_full + 8 * place, (sc >> 2) & 1, p.wait_ns))) continue;
                            w = (w + comb[my]) + (comb[kKeys + my] + comb[2 * kKeys + my]);
                            if (blk >= 0 && blk < p.num_blocks) {
                                float* at = p.scores + ((long long)blk * p.Hkv + it.h) * kBlock + key % kBlock;
                                *at = p.fresh || key >= it.x.first ? w : *at + w;
                            }
                        }
                    }
                    ++sc;
                }
                if (MODE == kSum) {
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(l_empty + 8 * (yc % kLseSlots));
                }
            }
            if (MODE == kWindow) {
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(l_empty + 8 * (ic % kLseSlots));
                continue;
            }
            // the quarters of a row. A warp whose wait ran out still meets the
            // others here, and all of them leave together.
            float2* comb = reinterpret_cast<float2*>(base + SM::kComb) + (ic & 1) * 2 * kQuarters * kKeys;
            if (!ok && lane == 0) failed[ic & 1] = 1;
#pragma unroll
            for (int t = 0; t < 2; ++t) comb[(t * kQuarters + quarter) * kKeys + my] = make_float2(m[t], sum[t]);
            asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
            if (failed[ic & 1]) {
                ok = false;
                break;
            }
            if (quarter < 2 && (quarter == 0 ? mine[0] : mine[1])) {
                const int t = quarter;  // this warp finishes tile t
                float2 q[kQuarters];
#pragma unroll
                for (int u = 0; u < kQuarters; ++u) q[u] = comb[(t * kQuarters + u) * kKeys + my];
                if (MODE == kLse) {
                    const float M = fmaxf(fmaxf(q[0].x, q[1].x), fmaxf(q[2].x, q[3].x));
                    const float v = M == -INFINITY ? 0.f : M;
                    const float l = (q[0].y * exp2f(q[0].x - v) + q[1].y * exp2f(q[1].x - v)) +
                                    (q[2].y * exp2f(q[2].x - v) + q[3].y * exp2f(q[3].x - v));
                    p.part[(long long)it.slot * kRows + t * kKeys + my] =
                        l == 0.f ? -INFINITY : M + log2f(l);
                } else {
                    const float w = (q[0].y + q[1].y) + (q[2].y + q[3].y);
                    const int key = it.row0 + t * kKeys + my;
                    const int blk = __ldg(p.tables + (long long)it.r * p.mbps + key / kBlock);
                    if (blk >= 0 && blk < p.num_blocks) {
                        float* at = p.scores + ((long long)blk * p.Hkv + it.h) * kBlock + key % kBlock;
                        *at = p.fresh || key >= it.x.first ? w : *at + w;
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

// For kSum: every row's log-sum-exp, a thread each, and its item counter back to
// zero.
__global__ void __launch_bounds__(kMergeThreads) window_merge_kernel(const WindowParams p) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.next = 0u;
    const long long share = __ldcg(p.begin + p.R);
    if (share == 0) return;
    const long long row = (long long)blockIdx.x * kMergeThreads + threadIdx.x;
    const int i = (int)(row / p.Hq), j = (int)(row % p.Hq);
    if (i < __ldg(p.query_start) || i >= __ldg(p.query_start + p.R)) return;
    int lo = 0, hi = p.R;  // query_start[lo] <= i < query_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.query_start + mid) <= i) lo = mid;
        else hi = mid;
    }
    const Request x = request_of(p, lo);
    if (x.m < 0) return;
    const int rb = (i - x.q0) / p.tokens, h = j / p.G;
    float v[1];
    merge_rows(row_parts(p, x, lo, rb, h, share), (i - x.q0 - rb * p.tokens) * p.G + j % p.G, v);
    p.nlse[((long long)h * p.T + i) * p.G + j % p.G] = v[0];
}

size_t lse_bytes(const mi_dims& D, int32_t total_q) { return ((size_t)total_q * D.Hq * 4 + 255) / 256 * 256; }

size_t begin_bytes(const mi_dims& D) { return ((size_t)(D.B + 1) * 8 + 255) / 256 * 256; }

size_t window_bytes(const mi_dims& D, int32_t total_q) {
    return 256 + begin_bytes(D) + lse_bytes(D, total_q) + slots(D.Hkv, D.Hq / D.Hkv, D.B, total_q) * kRows * 4;
}

bool window_sizes_ok(const mi_dims& D, int32_t total_q, int32_t max_query_len) {
    return total_q >= 0 && max_query_len >= 0 && (long long)total_q * D.Hq <= 0x7FFFFFFFLL &&
           (long long)max_query_len * D.Hq <= 0x7FFFFFFFLL;
}

template <int HD, int MODE>
bool launch_window(const CUtensorMap& tq, const CUtensorMap& tk, const WindowParams& p, cudaStream_t st) {
    static std::mutex mu;
    static CUcontext done[256] = {};
    if (!raise_smem(reinterpret_cast<const void*>(window_kernel<HD, MODE>), WinSmem<HD, MODE>::kTotal, done, mu)) return false;
    return launch_pdl(window_kernel<HD, MODE>, p.grid, kThreads, WinSmem<HD, MODE>::kTotal, st, tq, tk, p) == cudaSuccess;
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
    uint8_t* ws = static_cast<uint8_t*>(workspace) + 256;
    p.begin = reinterpret_cast<long long*>(ws);
    p.nlse = reinterpret_cast<float*>(ws += begin_bytes(D));
    p.part = reinterpret_cast<float*>(ws + lse_bytes(D, total_q));
    p.scores = scores;
    p.dev_err = dev_err;
    p.R = D.B;
    p.Hq = D.Hq;
    p.Hkv = D.Hkv;
    p.G = G;
    p.tokens = kRows / G;
    p.num_blocks = D.num_blocks;
    p.mbps = D.max_blocks_per_seq;
    p.T = total_q;
    p.max_q = max_query_len;
    p.fresh = fresh != 0;
    p.xt = 0;
    p.grid = sms < kMostBlocks ? sms : kMostBlocks;
    p.sl2 = scale * 1.4426950408889634f;
    // a scale of 0 weighs every key the same, and so does one that leaves
    // every logit far below 2^-24 (a masked logit times 0 would be NaN)
    if (p.sl2 == 0.f) p.sl2 = 1.2e-38f;
    p.wait_ns = test_wait_limit_ns();
    p.withhold = test_withhold_copy() ? 1 : 0;
    CUtensorMap tq, tk;
    // without queries the first map may name any tensor that holds a row of q:
    // kWindow still loads X for requests that have keys only, and no product of
    // it is used
    if (!make_tmap_q_group(&tq, total_q > 0 ? q : k_cache, total_q > 0 ? total_q : 1, D.Hq, HD, G, kRows / G * G) ||
        !make_tmap_kv_groups(&tk, k_cache, (long long)D.num_blocks * D.Hkv * kBlock, HD))
        return MI_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    const long long rows = (long long)total_q * D.Hq;
    const bool wide = HD == 128;
    // few enough rows stay resident while the keys stream
    const bool few = max_query_len <= kRows / G;
    p.xt = (long long)max_query_len * G <= kKeys ? 1 : 2;
    bool ok = wide ? launch_window<128, kLse>(tq, tk, p, st) : launch_window<64, kLse>(tq, tk, p, st);
    if (ok && !few)
        ok = launch_pdl(window_merge_kernel, (int)((rows + kMergeThreads) / kMergeThreads), kMergeThreads, 0, st, p) ==
             cudaSuccess;
    if (ok && few) ok = wide ? launch_window<128, kWindow>(tq, tk, p, st) : launch_window<64, kWindow>(tq, tk, p, st);
    if (ok && !few) ok = wide ? launch_window<128, kSum>(tq, tk, p, st) : launch_window<64, kSum>(tq, tk, p, st);
    return ok ? MI_OK : MI_ERR_CUDA;
}
