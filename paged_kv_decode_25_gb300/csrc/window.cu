// mi_paged_prefill_scores: the attention weight every cached token receives
// from many query tokens at once (the last tokens of a prompt, or all of it).
//
//   score[r][h][t] (+)= sum over query tokens i of request r with t <= pos_i
//                       and the G query heads j of h of 2^(x_ijt - lse_ij)
//
// Two launches, each computing the logits x once: window_lse_kernel reduces
// them over the keys of each row to the row's log-sum-exp, window_sum_kernel
// over the rows of each key to the key's weight. V is never read.
#include <cmath>

#include "batch.cuh"
#include "tiles.cuh"

namespace mi {
namespace {


struct WindowParams {
    const uint16_t* q;             // [T][Hq][HD]
    const uint16_t* k;             // [num_blocks][Hkv][16][HD]
    const int32_t* tables;         // [R][mbps]
    const int32_t* lens;           // [R]
    const int32_t* query_start;    // [R + 1]
    float* lse;                    // [T][Hq] base 2
    float* scores;                 // [num_blocks][Hkv][16]
    int32_t* dev_err;
    int R, Hq, Hkv, G, num_blocks, mbps, T, max_q, fresh;
    float sl2;
};

// Request r: n tokens, the last m of them with queries in rows q0 .. q0+m-1;
// first = n - m (negative: the rows before position 0 see nothing). A request
// whose bounds are bad has m = -1 and is left alone.
struct Request {
    int n, m, q0, first;
};

__device__ __forceinline__ Request request_of(const WindowParams& p, int r) {
    Request x;
    x.q0 = __ldg(p.query_start + r);
    const int q1 = __ldg(p.query_start + r + 1);
    x.m = q1 - x.q0;
    x.n = min(max(__ldg(p.lens + r), 0), p.mbps * kBlock);
    x.first = x.n - x.m;
    if (x.m < 0 || x.m > p.max_q) x.m = -1;
    return x;
}

template <int HD>
__device__ __forceinline__ const uint16_t* key_row(const WindowParams& p, int r, int h, int t, int n) {
    if (t >= n) return nullptr;
    const int blk = __ldg(p.tables + (long long)r * p.mbps + t / kBlock);
    if (blk < 0 || blk >= p.num_blocks) return nullptr;
    return p.k + (((long long)blk * p.Hkv + h) * kBlock + t % kBlock) * HD;
}

template <int HD>
__device__ __forceinline__ const uint16_t* query_row(const WindowParams& p, const Request& x, int h, int rho) {
    if (rho >= x.m * p.G) return nullptr;
    return p.q + ((long long)(x.q0 + rho / p.G) * p.Hq + (long long)h * p.G + rho % p.G) * HD;
}

template <int HD>
__global__ void __launch_bounds__(kTileThreads) window_lse_kernel(const WindowParams p) {
    __shared__ __align__(16) unsigned char qs[kTileRows * kPitch<HD>], ks[kTileRows * kPitch<HD>];
    __shared__ long long sums[flat_words(kTileThreads)];
    __shared__ uint32_t there;  // which of the tile's four key blocks are in the cache
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!starts_ascend(p.query_start, p.R, p.T)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
        return;
    }
    auto items = [&](int r) {
        const int m = request_of(p, r).m;
        return m > 0 ? (long long)p.Hkv * (((long long)m * p.G + kTileRows - 1) / kTileRows) : 0ll;
    };
    for (int r = blockIdx.x * kTileThreads + threadIdx.x; r < p.R; r += gridDim.x * kTileThreads) {
        const Request x = request_of(p, r);
        if (x.m < 0 || x.m > x.n) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
        if (__ldg(p.lens + r) > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
    }
    const long long total = flat_scan(p.R, items, sums);
    for (long long it = blockIdx.x; it < total; it += gridDim.x) {
        long long firstitem;
        const int r = flat_find(p.R, items, sums, it, firstitem);
        const Request x = request_of(p, r);
        const int tiles = (x.m * p.G + kTileRows - 1) / kTileRows;
        const int o = (int)(it - firstitem), h = o / tiles, rho0 = (o % tiles) * kTileRows;
        __syncthreads();
        load_tile<HD>(qs, [&](int i) { return query_row<HD>(p, x, h, rho0 + i); });
        __syncthreads();
        uint32_t a[HD / 16][4];
        load_a<HD>(a, smem_u32(qs), warp * 16, lane);
        const int row0 = rho0 + warp * 16 + (lane >> 2), row1 = row0 + 8;
        const int pos0 = x.first + row0 / p.G, pos1 = x.first + row1 / p.G;
        const int keys = min(x.n, x.first + min(x.m - 1, (rho0 + kTileRows - 1) / p.G) + 1);  // any row of the tile sees
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        for (int t0 = 0; t0 < keys; t0 += kTileRows) {
            __syncthreads();
            if (threadIdx.x < 32) {
                const int t = t0 + lane * kBlock;
                bool ok = false;
                if (lane < kTileRows / kBlock && t < x.n) {
                    const int blk = __ldg(p.tables + (long long)r * p.mbps + t / kBlock);
                    ok = blk >= 0 && blk < p.num_blocks;
                    if (!ok) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
                }
                const uint32_t msk = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) there = msk;
            }
            load_tile<HD>(ks, [&](int i) { return key_row<HD>(p, r, h, t0 + i, x.n); });
            __syncthreads();
            const uint32_t msk = there;
#pragma unroll
            for (int kb = 0; kb < kTileRows / kBlock; ++kb) {
                if (!((msk >> kb) & 1u)) continue;
                float c[2][4];
                product16<HD>(c, a, smem_u32(ks), kb * kBlock, lane);
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = t0 + kb * kBlock + t * 8 + 2 * (lane & 3) + (e & 1);
                        const bool keep = key <= (e < 2 ? pos0 : pos1);
                        c[t][e] = keep ? c[t][e] * p.sl2 : -INFINITY;
                        if (e < 2) x0 = fmaxf(x0, c[t][e]);
                        else x1 = fmaxf(x1, c[t][e]);
                    }
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
                l0 = l0 * exp2f(m0 - u0) + ((exp2f(c[0][0] - u0) + exp2f(c[0][1] - u0)) + (exp2f(c[1][0] - u0) + exp2f(c[1][1] - u0)));
                l1 = l1 * exp2f(m1 - u1) + ((exp2f(c[0][2] - u1) + exp2f(c[0][3] - u1)) + (exp2f(c[1][2] - u1) + exp2f(c[1][3] - u1)));
                m0 = n0;
                m1 = n1;
            }
        }
        // the four lanes of a row
#pragma unroll
        for (int sh = 1; sh < 4; sh <<= 1) {
            const float om0 = __shfl_xor_sync(0xffffffffu, m0, sh), ol0 = __shfl_xor_sync(0xffffffffu, l0, sh);
            const float om1 = __shfl_xor_sync(0xffffffffu, m1, sh), ol1 = __shfl_xor_sync(0xffffffffu, l1, sh);
            const float n0 = fmaxf(m0, om0), n1 = fmaxf(m1, om1);
            const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
            l0 = l0 * exp2f(m0 - u0) + ol0 * exp2f(om0 - u0);
            l1 = l1 * exp2f(m1 - u1) + ol1 * exp2f(om1 - u1);
            m0 = n0;
            m1 = n1;
        }
        // a row that sees no key gets +inf: every weight of it is 2^-inf = 0
        if ((lane & 3) == 0) {
            if (row0 < x.m * p.G)
                p.lse[(long long)(x.q0 + row0 / p.G) * p.Hq + h * p.G + row0 % p.G] = l0 > 0.f ? m0 + log2f(l0) : INFINITY;
            if (row1 < x.m * p.G)
                p.lse[(long long)(x.q0 + row1 / p.G) * p.Hq + h * p.G + row1 % p.G] = l1 > 0.f ? m1 + log2f(l1) : INFINITY;
        }
    }
}

template <int HD>
__global__ void __launch_bounds__(kTileThreads) window_sum_kernel(const WindowParams p) {
    __shared__ __align__(16) unsigned char qs[kTileRows * kPitch<HD>], ks[kTileRows * kPitch<HD>];
    __shared__ long long sums[flat_words(kTileThreads)];
    __shared__ float lses[kTileRows];
    __shared__ int poss[kTileRows];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!starts_ascend(p.query_start, p.R, p.T)) return;  // (reported by the first kernel)
    auto items = [&](int r) {
        const Request x = request_of(p, r);
        return x.m >= 0 ? (long long)p.Hkv * ((x.n + kTileRows - 1) / kTileRows) : 0ll;
    };
    const long long total = flat_scan(p.R, items, sums);
    for (long long it = blockIdx.x; it < total; it += gridDim.x) {
        long long firstitem;
        const int r = flat_find(p.R, items, sums, it, firstitem);
        const Request x = request_of(p, r);
        const int tiles = (x.n + kTileRows - 1) / kTileRows;
        const int o = (int)(it - firstitem), h = o / tiles, t0 = (o % tiles) * kTileRows;
        __syncthreads();
        load_tile<HD>(ks, [&](int i) { return key_row<HD>(p, r, h, t0 + i, x.n); });
        __syncthreads();
        uint32_t a[HD / 16][4];
        load_a<HD>(a, smem_u32(ks), warp * 16, lane);
        const int key0 = t0 + warp * 16 + (lane >> 2), key1 = key0 + 8;
        float w0 = 0.f, w1 = 0.f;
        // the first row that sees any key of the tile
        const int rows = x.m * p.G, from = max(0, t0 - x.first) * p.G / kTileRows * kTileRows;
        for (int rho0 = from; rho0 < rows; rho0 += kTileRows) {
            __syncthreads();
            load_tile<HD>(qs, [&](int i) { return query_row<HD>(p, x, h, rho0 + i); });
            if (threadIdx.x < kTileRows) {
                const int rho = rho0 + threadIdx.x;
                lses[threadIdx.x] = rho < rows ? p.lse[(long long)(x.q0 + rho / p.G) * p.Hq + h * p.G + rho % p.G] : INFINITY;
                poss[threadIdx.x] = rho < rows ? x.first + rho / p.G : -1;
            }
            __syncthreads();
#pragma unroll
            for (int rb = 0; rb < kTileRows / 16; ++rb) {
                float c[2][4];
                product16<HD>(c, a, smem_u32(qs), rb * 16, lane);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = rb * 16 + t * 8 + 2 * (lane & 3) + (e & 1);
                        const float w = (e < 2 ? key0 : key1) <= poss[i] ? exp2f(c[t][e] * p.sl2 - lses[i]) : 0.f;
                        if (e < 2) w0 += w;
                        else w1 += w;
                    }
            }
        }
#pragma unroll
        for (int sh = 1; sh < 4; sh <<= 1) {
            w0 += __shfl_xor_sync(0xffffffffu, w0, sh);
            w1 += __shfl_xor_sync(0xffffffffu, w1, sh);
        }
        if ((lane & 3) == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = e ? key1 : key0;
                if (t >= x.n) continue;
                const int blk = __ldg(p.tables + (long long)r * p.mbps + t / kBlock);
                if (blk < 0 || blk >= p.num_blocks) continue;
                float* at = p.scores + ((long long)blk * p.Hkv + h) * kBlock + t % kBlock;
                const float w = e ? w1 : w0;
                *at = p.fresh || t >= x.first ? w : *at + w;
            }
        }
    }
}

size_t window_bytes(const mi_dims& D, int32_t total_q) {
    return ((size_t)total_q * D.Hq * 4 + 255) / 256 * 256 + 256;
}

bool window_sizes_ok(const mi_dims& D, int32_t total_q, int32_t max_query_len) {
    return total_q >= 0 && max_query_len >= 0 && (long long)total_q * D.Hq <= 0x7FFFFFFFLL &&
           (long long)max_query_len * D.Hq <= 0x7FFFFFFFLL;
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
    WindowParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_cache);
    p.tables = block_tables;
    p.lens = context_lens;
    p.query_start = query_start;
    p.lse = static_cast<float*>(workspace);
    p.scores = scores;
    p.dev_err = dev_err;
    p.R = D.B;
    p.Hq = D.Hq;
    p.Hkv = D.Hkv;
    p.G = D.Hq / D.Hkv;
    p.num_blocks = D.num_blocks;
    p.mbps = D.max_blocks_per_seq;
    p.T = total_q;
    p.max_q = max_query_len;
    p.fresh = fresh != 0;
    p.sl2 = scale * 1.4426950408889634f;
    cudaStream_t st = (cudaStream_t)stream;
    const bool wide = D.head_dim == 128;
    const int grid = 4 * sms;
    if (launch_pdl(wide ? window_lse_kernel<128> : window_lse_kernel<64>, grid, kTileThreads, 0, st, p) != cudaSuccess)
        return MI_ERR_CUDA;
    return launch_pdl(wide ? window_sum_kernel<128> : window_sum_kernel<64>, grid, kTileThreads, 0, st, p) == cudaSuccess
               ? MI_OK
               : MI_ERR_CUDA;
}
