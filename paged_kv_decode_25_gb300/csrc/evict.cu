// mi_paged_kv_evict: a smaller paged cache from accumulated attention weights.
//
// For request b and KV head h with n tokens, a budget k = min(n, budgets[b])
// and r = min(recent, k), the kept tokens are the newest r and, of the n - r
// older ones, the k - r with the largest scores (equal scores: the lower
// index first). They keep their order and become tokens 0 .. k-1 of the
// destination table. Each KV head keeps its own tokens: a block holds every
// head's rows of 16 token indices, and nothing else ties the heads together.
//
// Two launches:
//   * evict_select_kernel finds the (k - r)-th largest score of every (b, h)
//     by a radix select over an order-preserving 32-bit key, and writes the
//     kept older tokens' indices in ascending order. Where the (b, h) do not
//     fill the GPU, a cluster of up to 8 blocks shares one: each holds a
//     stretch of the tokens and adds up the others' digit counts through
//     distributed shared memory (16 (b, h) of 30,000 to 120,000 tokens: 22 us,
//     with one block each 73);
//   * evict_move_kernel copies the kept rows of K and V and their scores.
// Both only move bytes: the floor is the scores once, the kept rows in and
// out. 64 requests of 2,000 to 8,192 tokens cut to 2,048: the selection 22 us
// (the keys are read from shared memory three times more, the digit counts are
// atomics on a few hot bins), the move 172 us for 1.08 GB (6.3 TB/s).
// In place each (request, head) moves in steps of 64 rows by one block, so that
// rows are read before they are overwritten: as fast where there are hundreds
// of them (512: 175 us), but latency by latency where there are few (4 e4m3
// requests of 30,000 to 120,000 with 4 heads: 189 us, out of place 12).
#include <algorithm>
#include <mutex>

#include "batch.cuh"

namespace mi {
namespace {

constexpr int kBins = 2048;                // digits of 11, 11 and 10 bits
constexpr int kSelKeys = 24576;            // keys a block holds in shared memory (96 KB: two blocks an SM)
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;              // destination rows per work item

struct EvictParams {
    uint8_t* k;                    // [num_blocks][Hkv][16] rows of row bytes
    uint8_t* v;
    float* scores;                 // [num_blocks][Hkv][16]
    const int32_t* tables;         // [B][mbps]
    const int32_t* lens;           // [B]
    const int32_t* budgets;        // [B]
    const int32_t* dst;            // [B][mbps]
    int32_t* new_lens;             // [B]
    int32_t* list;                 // [B][Hkv][mbps * 16]: kept older tokens, ascending
    int32_t* dev_err;
    int B, Hkv, num_blocks, mbps, recent, in_place;
};

// What request b keeps: n tokens now, `kept` of them afterwards, the last
// `tail` of which are its newest and the first `heavy` chosen by score among
// tokens 0 .. old-1. A request that keeps everything has no chosen tokens.
struct Share {
    int n, kept, tail, heavy, old;
};

__device__ __forceinline__ Share share_of(const EvictParams& p, int b) {
    Share s;
    s.n = min(max(__ldg(p.lens + b), 0), p.mbps * kBlock);
    s.kept = min(s.n, max(__ldg(p.budgets + b), 0));
    s.tail = s.kept == s.n ? s.n : min(p.recent, s.kept);
    s.heavy = s.kept - s.tail;
    s.old = s.n - s.tail;
    return s;
}

// Monotone in the score, as an unsigned number: NaN lowest, then -inf up to
// +inf, the two zeros equal.
__device__ __forceinline__ uint32_t score_key(float x) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    if (u == 0x80000000u) u = 0u;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Keys of tokens 4 * t4 .. 4 * t4 + 3 (0 for a block id outside the cache).
__device__ __forceinline__ void load_keys(const EvictParams& p, int b, int h, int t4, uint32_t (&key)[4], bool report) {
    const int blk = __ldg(p.tables + (long long)b * p.mbps + (t4 >> 2));
    if (blk < 0 || blk >= p.num_blocks) {
        if (report) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
        key[0] = key[1] = key[2] = key[3] = 0u;
        return;
    }
    const float4 s = *reinterpret_cast<const float4*>(p.scores + ((long long)blk * p.Hkv + h) * kBlock + (t4 & 3) * 4);
    key[0] = score_key(s.x);
    key[1] = score_key(s.y);
    key[2] = score_key(s.z);
    key[3] = score_key(s.w);
}

// Exclusive sum over the block; `total` is the sum. wsum: 32 words.
__device__ __forceinline__ uint32_t block_sum_before(uint32_t v, uint32_t* wsum, uint32_t& total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the previous use of wsum is over
    if (lane == 31) wsum[wid] = x;
    __syncthreads();
    if (wid == 0) {
        uint32_t t = lane < nw ? wsum[lane] : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        wsum[lane] = t;
    }
    __syncthreads();
    total = wsum[31];
    return (wid ? wsum[wid - 1] : 0u) + x - v;
}

// A word of the block `rank` of the cluster, at this block's shared address.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t* mine, uint32_t rank) {
    uint32_t addr, v;  // (volatile orders it among the cluster barriers and leaves the loads in flight together)
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void cluster_store(uint32_t* mine, uint32_t rank, uint32_t v) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster of RANKS blocks per (b, h); block `rank` of it takes the
// stretch of quads (four tokens) [rank * share, (rank + 1) * share). Its keys
// stay in shared memory (`held` of them; the rest is read again). Every block
// of a cluster takes the same way through the kernel.
template <int RANKS, int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const EvictParams p, int held) {
    constexpr int kPer = kBins / THREADS;  // bins a thread counts (a block alone)
    extern __shared__ uint4 keys[];  // [held / 4]
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wsum[32];
    __shared__ uint32_t found[2];
    __shared__ uint32_t counts[2];
    __shared__ uint32_t sums[RANKS > 1 ? kBins / RANKS + 1 : 1], totals[RANKS];
    pdl_wait();
    pdl_trigger();
    const int unit = blockIdx.x / RANKS, rank = blockIdx.x % RANKS;
    const int b = unit / p.Hkv, h = unit % p.Hkv, tid = threadIdx.x;
    const Share s = share_of(p, b);
    if (h == 0 && rank == 0 && tid == 0) {
        p.new_lens[b] = s.kept;
        if (__ldg(p.lens + b) > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
    }
    if (s.heavy == 0) return;
    const int all = (s.old + 3) / 4, share = (all + RANKS - 1) / RANKS;
    const int q0 = min(all, rank * share), quads = min(all, q0 + share) - q0;
    auto quad = [&](int i, bool first) -> uint4 {  // the keys of quad q0 + i; 0 past the older tokens
        if (!first && 4 * i < held) return keys[i];
        uint32_t k[4];
        load_keys(p, b, h, q0 + i, k, first);
        const uint4 v = make_uint4(k[0], k[1], k[2], k[3]);
        if (first && 4 * i < held) keys[i] = v;
        return v;
    };
    uint32_t prefix = 0, need = (uint32_t)s.heavy;  // of the tokens whose key starts with `prefix`, take the top `need`
    int low = 32;                                   // key bits below the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, up = low;
        low -= bits;
        for (int i = tid; i < kBins; i += THREADS) hist[i] = 0u;
        __syncthreads();
        for (int i = tid; i < quads; i += THREADS) {
            const uint4 v = quad(i, pass == 0);
            const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * (q0 + i) + e < s.old && (pass == 0 || (key[e] >> up) == prefix))
                    atomicAdd(&hist[(key[e] >> low) & ((1u << bits) - 1u)], 1u);
        }
        const int top = (1 << bits) - 1;  // bins are taken from the top down
        if constexpr (RANKS == 1) {
            __syncthreads();
            uint32_t c[kPer], n = 0;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int bin = top - kPer * tid - u;
                c[u] = bin >= 0 ? hist[bin] : 0u;
                n += c[u];
            }
            uint32_t total;
            uint32_t before = block_sum_before(n, wsum, total);
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                if (before < need && need <= before + c[u]) {
                    found[0] = (uint32_t)(top - kPer * tid - u);
                    found[1] = before;
                }
                before += c[u];
            }
        } else {
            // each block adds up a RANKS-th of the bins over the cluster and
            // hands every block its total; then all look into the part that
            // holds the digit (with every block adding up all bins, the
            // remote loads were half the kernel: 59 us a step against 38, for 4 x 4 of 30,000 to 120,000 tokens)
            constexpr int kOwn = kBins / RANKS;
            static_assert(kOwn <= THREADS, "a thread per bin");
            cluster_sync();
            uint32_t c = 0, total;
            const int bin = top - rank * kOwn - tid;
            if (tid < kOwn && bin >= 0) {
                uint32_t part[RANKS];
#pragma unroll
                for (int r = 0; r < RANKS; ++r) part[r] = cluster_word(hist + bin, r);
#pragma unroll
                for (int r = 0; r < RANKS; ++r) c += part[r];
            }
            const uint32_t before = block_sum_before(c, wsum, total);
            if (tid < kOwn) sums[tid] = before;
            if (tid == 0) sums[kOwn] = total;
            if (tid < RANKS) cluster_store(totals + rank, tid, total);
            cluster_sync();
            int owner = 0;
            uint32_t base = 0;
            while (owner < RANKS - 1 && need > base + totals[owner]) base += totals[owner++];
            if (tid < kOwn) {
                const uint32_t lo = base + cluster_word(sums + tid, owner), hi = base + cluster_word(sums + tid + 1, owner);
                if (lo < need && need <= hi) {
                    found[0] = (uint32_t)(top - owner * kOwn - tid);
                    found[1] = lo;
                }
            }
        }
        __syncthreads();
        prefix = (prefix << bits) | found[0];
        need -= found[1];
        __syncthreads();
    }
    // every token with a larger key, and the first `need` of those with the
    // key itself, in ascending order
    uint32_t above = 0, equal = 0;  // in the stretches before this one, then seen so far
    if (RANKS > 1) {
        uint32_t gt = 0, eq = 0;
        for (int i = tid; i < quads; i += THREADS) {
            const uint4 v = quad(i, false);
            const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (4 * (q0 + i) + e >= s.old) continue;
                gt += key[e] > prefix;
                eq += key[e] == prefix;
            }
        }
        uint32_t gt_all, eq_all;
        block_sum_before(gt, wsum, gt_all);
        block_sum_before(eq, wsum, eq_all);
        if (tid == 0) {
            counts[0] = gt_all;
            counts[1] = eq_all;
        }
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            above += cluster_word(counts, r);
            equal += cluster_word(counts + 1, r);
        }
        cluster_sync();  // no block leaves while another reads its shared memory
    }
    int32_t* list = p.list + ((long long)b * p.Hkv + h) * p.mbps * kBlock;
    for (int base = 0; base < quads; base += THREADS) {
        const int i = base + tid;
        uint32_t key[4] = {0u, 0u, 0u, 0u};
        uint32_t gt = 0, eq = 0;
        if (i < quads) {
            const uint4 v = quad(i, false);
            key[0] = v.x;
            key[1] = v.y;
            key[2] = v.z;
            key[3] = v.w;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (4 * (q0 + i) + e >= s.old) continue;
                gt += key[e] > prefix;
                eq += key[e] == prefix;
            }
        }
        uint32_t total;
        const uint32_t before = block_sum_before((gt << 16) | eq, wsum, total);
        uint32_t g = above + (before >> 16), q = equal + (before & 0xFFFFu);
        if (i < quads) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * (q0 + i) + e;
                if (t >= s.old) continue;
                if (key[e] > prefix) {
                    list[g + min(q, need)] = t;
                    ++g;
                } else if (key[e] == prefix) {
                    if (q < need) list[g + q] = t;
                    ++q;
                }
            }
        }
        above += total >> 16;
        equal += total & 0xFFFFu;
    }
}

// Rows of the cache (in units of one token of one head) that destination
// token i of (b, h) comes from and goes to; -1 for a block id outside the cache.
__device__ __forceinline__ int2 row_move(const EvictParams& p, const Share& s, int b, int h, int i) {
    const int t = i < s.heavy ? p.list[((long long)b * p.Hkv + h) * p.mbps * kBlock + i] : s.old + (i - s.heavy);
    const int from = __ldg(p.tables + (long long)b * p.mbps + t / kBlock);
    const int to = __ldg(p.dst + (long long)b * p.mbps + i / kBlock);
    const bool ok_f = from >= 0 && from < p.num_blocks, ok_t = to >= 0 && to < p.num_blocks;
    if (!ok_f || !ok_t) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
    return make_int2(ok_f && ok_t ? (from * p.Hkv + h) * kBlock + t % kBlock : -1,
                     ok_f && ok_t ? (to * p.Hkv + h) * kBlock + i % kBlock : -1);
}

// One work item: destination rows i0 .. i0 + 63 of (b, h). V16: 16-byte
// vectors of a row.
template <int V16>
__device__ __forceinline__ void move_rows(const EvictParams& p, const Share& s, int b, int h, int i0, int2* rows) {
    constexpr int kVecs = kMoveRows * V16 / kMoveThreads;  // per thread and cache
    const int tid = threadIdx.x;
    float sc = 0.f;
    __syncthreads();  // the previous item is done with `rows` (and, in place, has written what it moves)
    if (tid < kMoveRows) {
        const int2 m = i0 + tid < s.kept ? row_move(p, s, b, h, i0 + tid) : make_int2(-1, -1);
        rows[tid] = m;
        if (m.x >= 0) sc = p.scores[m.x];
    }
    __syncthreads();
    uint4 a[kVecs], c[kVecs];
    int2 m[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kMoveThreads + tid;
        m[u] = rows[i / V16];
        if (m[u].x >= 0) {
            a[u] = reinterpret_cast<const uint4*>(p.k)[(long long)m[u].x * V16 + i % V16];
            c[u] = reinterpret_cast<const uint4*>(p.v)[(long long)m[u].x * V16 + i % V16];
        }
    }
    // in place, a row may land on one that another thread of this item still
    // has to read; rows of later items lie above everything written here
    if (p.in_place) __syncthreads();
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kMoveThreads + tid;
        if (m[u].x >= 0) {
            reinterpret_cast<uint4*>(p.k)[(long long)m[u].y * V16 + i % V16] = a[u];
            reinterpret_cast<uint4*>(p.v)[(long long)m[u].y * V16 + i % V16] = c[u];
        }
    }
    if (tid < kMoveRows && rows[tid].x >= 0) p.scores[rows[tid].y] = sc;
}

template <int V16>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
    __shared__ long long sums[flat_words(kMoveThreads)];
    __shared__ int2 rows[kMoveRows];
    // lengths and budgets were there before the selection: the plan is made
    // while it runs
    if (p.in_place) {
        // a kept row never moves up, so items in ascending order never
        // overwrite a row that is still to be read: one block per (b, h)
        const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
        const Share s = share_of(p, b);
        pdl_wait();
        pdl_trigger();
        if (s.kept == s.n) return;
        for (int i0 = 0; i0 < s.kept; i0 += kMoveRows) move_rows<V16>(p, s, b, h, i0, rows);
        return;
    }
    auto items = [&](int b) { return (long long)p.Hkv * ((share_of(p, b).kept + kMoveRows - 1) / kMoveRows); };
    const long long total = flat_scan(p.B, items, sums);
    pdl_wait();
    pdl_trigger();
    for (long long x = blockIdx.x; x < total; x += gridDim.x) {
        long long first;
        const int b = flat_find(p.B, items, sums, x, first);
        const Share s = share_of(p, b);
        const int per = (s.kept + kMoveRows - 1) / kMoveRows;
        const int o = (int)(x - first);
        move_rows<V16>(p, s, b, o / per, (o % per) * kMoveRows, rows);
    }
}

size_t list_bytes(const mi_dims& D) {
    return ((size_t)D.B * D.Hkv * D.max_blocks_per_seq * kBlock * 4 + 255) / 256 * 256;
}

template <int RANKS, int THREADS>
bool launch_select(const EvictParams& p, int units, int held, cudaStream_t st) {
    static std::mutex mu;
    static CUcontext done[256] = {};
    auto* kernel = evict_select_kernel<RANKS, THREADS>;
    return raise_smem(reinterpret_cast<const void*>(kernel), kSelKeys * 4, done, mu) &&
           launch_cluster(kernel, units * RANKS, THREADS, held * 4, RANKS, st, p, held) == cudaSuccess;
}

mi_status evict(const mi_dims* dims, void* k_cache, void* v_cache, float* scores, const int32_t* block_tables,
                const int32_t* context_lens, const int32_t* budgets, int32_t recent, const int32_t* dst_tables,
                int32_t* new_lens, void* workspace, size_t workspace_bytes, int32_t* dev_err, mi_stream_t stream,
                int elem) {
    const mi_status ds = check_paged_dims(dims);
    if (ds != MI_OK) return ds;
    const mi_dims D = *dims;
    if (recent < 0) return MI_ERR_INVALID_ARG;
    if (D.B == 0) return MI_OK;
    if (!k_cache || !v_cache || !scores || !block_tables || !context_lens || !budgets || !dst_tables || !new_lens ||
        !workspace)
        return MI_ERR_INVALID_ARG;
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(scores, 16) || !aligned_to(workspace, 16) ||
        !aligned_to(block_tables, 4) || !aligned_to(context_lens, 4) || !aligned_to(budgets, 4) ||
        !aligned_to(dst_tables, 4) || !aligned_to(new_lens, 4))
        return MI_ERR_INVALID_ARG;
    if (workspace_bytes < list_bytes(D)) return MI_ERR_INVALID_ARG;
    // every block reads the lengths, budgets and tables while one of them writes new_lens
    const size_t lens_bytes = (size_t)D.B * 4, table_bytes = lens_bytes * D.max_blocks_per_seq;
    if (overlaps(new_lens, lens_bytes, context_lens, lens_bytes) || overlaps(new_lens, lens_bytes, budgets, lens_bytes) ||
        overlaps(new_lens, lens_bytes, block_tables, table_bytes) || overlaps(new_lens, lens_bytes, dst_tables, table_bytes))
        return MI_ERR_INVALID_ARG;
    if (dst_tables != block_tables && overlaps(dst_tables, table_bytes, block_tables, table_bytes))
        return MI_ERR_INVALID_ARG;
    if ((long long)D.B * D.Hkv > 0x7FFFFFFFLL / 8) return MI_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return MI_ERR_CUDA;
    EvictParams p;
    p.k = static_cast<uint8_t*>(k_cache);
    p.v = static_cast<uint8_t*>(v_cache);
    p.scores = scores;
    p.tables = block_tables;
    p.lens = context_lens;
    p.budgets = budgets;
    p.dst = dst_tables;
    p.new_lens = new_lens;
    p.list = static_cast<int32_t*>(workspace);
    p.dev_err = dev_err;
    p.B = D.B;
    p.Hkv = D.Hkv;
    p.num_blocks = D.num_blocks;
    p.mbps = D.max_blocks_per_seq;
    p.recent = recent;
    p.in_place = dst_tables == block_tables ? 1 : 0;
    cudaStream_t st = (cudaStream_t)stream;
    const int units = D.B * D.Hkv;
    // blocks per (b, h): one where they fill the GPU, else up to 8 with at
    // least 2,048 of the longest request's tokens each
    const long long longest = (long long)D.max_blocks_per_seq * kBlock;
    int ranks = 1;
    while (ranks < 8 && 2LL * ranks * units <= 2LL * sms && longest / (2 * ranks) >= 2048) ranks *= 2;
    const long long stretch = (longest / 4 + ranks - 1) / ranks * 4 + 4;
    const int held = (int)(stretch < kSelKeys ? (stretch + 3) / 4 * 4 : kSelKeys);
    const bool sel = ranks == 1   ? launch_select<1, 512>(p, units, held, st)
                     : ranks == 2 ? launch_select<2, 1024>(p, units, held, st)
                     : ranks == 4 ? launch_select<4, 1024>(p, units, held, st)
                                  : launch_select<8, 1024>(p, units, held, st);
    if (!sel) return MI_ERR_CUDA;
    const int grid = p.in_place ? units : 8 * sms;
    cudaError_t e;
    switch (D.head_dim * elem / 16) {
        case 4: e = launch_pdl(evict_move_kernel<4>, grid, kMoveThreads, 0, st, p); break;
        case 8: e = launch_pdl(evict_move_kernel<8>, grid, kMoveThreads, 0, st, p); break;
        default: e = launch_pdl(evict_move_kernel<16>, grid, kMoveThreads, 0, st, p); break;
    }
    return e == cudaSuccess ? MI_OK : MI_ERR_CUDA;
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_paged_kv_evict_workspace_bytes(const mi_dims* dims) {
    return mi::check_paged_dims(dims) == MI_OK ? mi::list_bytes(*dims) : 0;
}

extern "C" mi_status mi_paged_kv_evict(const mi_dims* dims, void* k_cache, void* v_cache, float* scores,
                                       const int32_t* block_tables, const int32_t* context_lens,
                                       const int32_t* budgets, int32_t recent, const int32_t* dst_tables,
                                       int32_t* new_lens, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                       mi_stream_t stream) {
    return mi::evict(dims, k_cache, v_cache, scores, block_tables, context_lens, budgets, recent, dst_tables, new_lens,
                     workspace, workspace_bytes, dev_err, stream, 2);
}

extern "C" mi_status mi_paged_kv_evict_fp8(const mi_dims* dims, void* k_cache, void* v_cache, float* scores,
                                           const int32_t* block_tables, const int32_t* context_lens,
                                           const int32_t* budgets, int32_t recent, const int32_t* dst_tables,
                                           int32_t* new_lens, void* workspace, size_t workspace_bytes,
                                           int32_t* dev_err, mi_stream_t stream) {
    return mi::evict(dims, k_cache, v_cache, scores, block_tables, context_lens, budgets, recent, dst_tables, new_lens,
                     workspace, workspace_bytes, dev_err, stream, 1);
}
