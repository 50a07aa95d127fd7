// mi_paged_decode_attention_prefix: one decode step of a batch whose requests
// share prefixes, each prefix's keys and values read once for all of them.
//
// Request b of group g attends to the prefix's tokens followed by its own.
// The softmax over the two parts is put together from their (output,
// log-sum-exp) pairs, so the parts are computed apart:
//   * prefix_kernel: the group's queries against the prefix, as one tall
//     matrix of (request, head) rows per KV head: a staged K / V tile serves
//     every request of the group;
//   * the decode kernel (decode.cu) over the requests' own blocks, which
//     merges the prefix's partial results into each row as it finishes it.
//
// The rows of (group, KV head) are cut into tiles of whole requests, the
// prefix's blocks into equal splits; a (group, tile, split, head) is a work
// item and writes one slot of partial results. Every block finds the items
// from the lengths by itself; the split length is such that the whole grid
// has about one item each.
#include <cmath>

#include "batch.cuh"
#include "decode.cuh"
#include "tiles.cuh"

namespace mi {
namespace {

constexpr int kMinSplit = 8;     // blocks: a shorter split does not pay for its partial results
constexpr int kSplitStep = 4;    // a split is whole 64-key tiles

struct PrefixParams {
    const uint16_t* q;             // [B][Hq][HD]
    const uint16_t* k;             // [num_blocks][Hkv][16][HD]
    const uint16_t* v;
    const int32_t* tables;         // [P][mbps]
    const int32_t* lens;           // [P]
    const int32_t* starts;         // [P + 1]
    int4* rows;                    // [B] see DecodeExt
    float* part;
    float* part_lse;
    int32_t* dev_err;
    int P, B, Hq, Hkv, G, num_blocks, mbps, tile_rows, target;
    float sl2;
};

__device__ __forceinline__ int prefix_tokens(const PrefixParams& p, int g) {
    return min(max(__ldg(p.lens + g), 0), p.mbps * kBlock);
}
__device__ __forceinline__ int prefix_blocks(const PrefixParams& p, int g) {
    return (prefix_tokens(p, g) + kBlock - 1) / kBlock;
}
// Tiles of group g's rows; a tile holds per = tile_rows / G whole requests.
__device__ __forceinline__ int group_tiles(const PrefixParams& p, int g) {
    const int per = p.tile_rows / p.G;
    return (__ldg(p.starts + g + 1) - __ldg(p.starts + g) + per - 1) / per;
}

// Blocks per split, the same for every group.
__device__ __forceinline__ int split_blocks(long long total_blocks, int target) {
    const long long even = (total_blocks + target - 1) / target;
    const long long up = (even + kSplitStep - 1) / kSplitStep * kSplitStep;
    return (int)(up < kMinSplit ? kMinSplit : up > (1 << 27) ? 1 << 27 : up);  // a table has fewer blocks than 2^27
}

template <int HD>
__global__ void __launch_bounds__(kTileThreads) prefix_kernel(const PrefixParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char* qs = smem;
    unsigned char* ks = qs + kTileRows * kPitch<HD>;
    unsigned char* vs = ks + kTileRows * kPitch<HD>;
    __shared__ long long sums[flat_words(kTileThreads)];
    __shared__ uint32_t there;  // which of the tile's four key blocks are in the cache
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int gtid = blockIdx.x * kTileThreads + tid, nthreads = gridDim.x * kTileThreads;
    if (!starts_ascend(p.starts, p.P, p.B)) {
        // no request's prefix is known
        if (gtid == 0) raise_err(p.dev_err, MI_DEVERR_BAD_QUERY);
        for (int b = gtid; b < p.B; b += nthreads) p.rows[b] = make_int4(0, 0, 0, 0);
        return;
    }
    const long long cost = flat_scan(
        p.P, [&](int g) { return (long long)p.Hkv * group_tiles(p, g) * prefix_blocks(p, g); }, sums);
    const int step = split_blocks(cost, p.target);
    auto items = [&](int g) {
        return (long long)p.Hkv * group_tiles(p, g) * ((prefix_blocks(p, g) + step - 1) / step);
    };
    __syncthreads();
    const long long total = flat_scan(p.P, items, sums);
    for (int g = gtid; g < p.P; g += nthreads)
        if (__ldg(p.lens + g) > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
    // each request's slots; those outside every group have none
    const int per = p.tile_rows / p.G, b_first = __ldg(p.starts), b_last = __ldg(p.starts + p.P);
    for (int b = gtid; b < p.B; b += nthreads) {
        int4 at = make_int4(0, 0, 0, 0);
        if (b >= b_first && b < b_last) {
            int lo = 0, hi = p.P;  // starts[lo] <= b < starts[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.starts + mid) <= b) lo = mid;
                else hi = mid;
            }
            const int splits = (prefix_blocks(p, lo) + step - 1) / step;
            if (splits > 0) {
                long long first = sums[lo / ((p.P + kTileThreads - 1) / kTileThreads)];
                for (int g = lo / ((p.P + kTileThreads - 1) / kTileThreads) * ((p.P + kTileThreads - 1) / kTileThreads); g < lo; ++g)
                    first += items(g);
                const int i = b - __ldg(p.starts + lo);
                at = make_int4((int)first + (i / per) * splits * p.Hkv, splits, (i % per) * p.G, 0);
            }
        }
        p.rows[b] = at;
    }
    for (long long it = blockIdx.x; it < total; it += gridDim.x) {
        long long first;
        const int g = flat_find(p.P, items, sums, it, first);
        const int n = prefix_tokens(p, g), nblk = (n + kBlock - 1) / kBlock, splits = (nblk + step - 1) / step;
        const int o = (int)(it - first), h = o % p.Hkv, s = o / p.Hkv % splits, tile = o / p.Hkv / splits;
        const int b0 = __ldg(p.starts + g) + tile * per, b1 = min(__ldg(p.starts + g + 1), b0 + per);
        const int nrows = (b1 - b0) * p.G;
        const int t_end = (int)min((long long)n, (long long)(s + 1) * step * kBlock);
        __syncthreads();
        load_tile<HD>(qs, [&](int i) {
            return i < nrows ? p.q + ((long long)(b0 + i / p.G) * p.Hq + (long long)h * p.G + i % p.G) * HD : nullptr;
        });
        __syncthreads();
        uint32_t a[HD / 16][4];
        load_a<HD>(a, smem_u32(qs), warp * 16, lane);
        float acc[HD / 8][4];
#pragma unroll
        for (int t = 0; t < HD / 8; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        for (int t0 = s * step * kBlock; t0 < t_end; t0 += kTileRows) {
            __syncthreads();
            if (warp == 0) {
                const int t = t0 + lane * kBlock;
                bool ok = false;
                if (lane < kTileRows / kBlock && t < t_end) {
                    const int blk = __ldg(p.tables + (long long)g * p.mbps + t / kBlock);
                    ok = blk >= 0 && blk < p.num_blocks;
                    if (!ok) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
                }
                const uint32_t msk = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) there = msk;
            }
            // keys past the prefix's end may hold any bits: zeroed here
            auto row_of = [&](int i) -> long long {
                if (t0 + i >= n) return -1;
                const int blk = __ldg(p.tables + (long long)g * p.mbps + (t0 + i) / kBlock);
                return blk >= 0 && blk < p.num_blocks ? (((long long)blk * p.Hkv + h) * kBlock + i % kBlock) * HD : -1;
            };
            load_tile<HD>(ks, [&](int i) { const long long r = row_of(i); return r >= 0 ? p.k + r : nullptr; });
            load_tile<HD>(vs, [&](int i) { const long long r = row_of(i); return r >= 0 ? p.v + r : nullptr; });
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
                        c[t][e] = key < n ? c[t][e] * p.sl2 : -INFINITY;
                        if (e < 2) x0 = fmaxf(x0, c[t][e]);
                        else x1 = fmaxf(x1, c[t][e]);
                    }
#pragma unroll
                for (int sh = 1; sh < 4; sh <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, sh));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, sh));
                }
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
                const float f0 = exp2f(m0 - u0), f1 = exp2f(m1 - u1);
                m0 = n0;
                m1 = n1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    c[t][0] = exp2f(c[t][0] - u0);
                    c[t][1] = exp2f(c[t][1] - u0);
                    c[t][2] = exp2f(c[t][2] - u1);
                    c[t][3] = exp2f(c[t][3] - u1);
                }
                l0 = l0 * f0 + ((c[0][0] + c[0][1]) + (c[1][0] + c[1][1]));
                l1 = l1 * f1 + ((c[0][2] + c[0][3]) + (c[1][2] + c[1][3]));
#pragma unroll
                for (int t = 0; t < HD / 8; ++t) {
                    acc[t][0] *= f0;
                    acc[t][1] *= f0;
                    acc[t][2] *= f1;
                    acc[t][3] *= f1;
                }
                const uint32_t p0 = pack_bf16x2(c[0][0], c[0][1]), p1 = pack_bf16x2(c[0][2], c[0][3]);
                const uint32_t p2 = pack_bf16x2(c[1][0], c[1][1]), p3 = pack_bf16x2(c[1][2], c[1][3]);
#pragma unroll
                for (int d = 0; d < HD / 16; ++d) {
                    uint32_t v0, v1, v2, v3;
                    ldsm_x4_trans(smem_u32(vs) + (kb * kBlock + ((lane >> 3) & 1) * 8 + (lane & 7)) * kPitch<HD> +
                                      d * 32 + (lane >> 4) * 16,
                                  v0, v1, v2, v3);
                    mma_bf16_16816(acc[2 * d], p0, p1, p2, p3, v0, v1);
                    mma_bf16_16816(acc[2 * d + 1], p0, p1, p2, p3, v2, v3);
                }
            }
        }
#pragma unroll
        for (int sh = 1; sh < 4; sh <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
            l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
        }
        const int r0 = warp * 16 + (lane >> 2), r1 = r0 + 8;
        const float i0 = l0 > 0.f ? 1.f / l0 : 0.f, i1 = l1 > 0.f ? 1.f / l1 : 0.f;
        float* o0 = p.part + (it * p.tile_rows + r0) * HD + 2 * (lane & 3);
        float* o1 = o0 + 8 * HD;
#pragma unroll
        for (int t = 0; t < HD / 8; ++t) {
            if (r0 < nrows) *reinterpret_cast<float2*>(o0 + 8 * t) = make_float2(acc[t][0] * i0, acc[t][1] * i0);
            if (r1 < nrows) *reinterpret_cast<float2*>(o1 + 8 * t) = make_float2(acc[t][2] * i1, acc[t][3] * i1);
        }
        if ((lane & 3) == 0) {
            if (r0 < nrows) p.part_lse[it * p.tile_rows + r0] = l0 > 0.f ? m0 + log2f(l0) : -INFINITY;
            if (r1 < nrows) p.part_lse[it * p.tile_rows + r1] = l1 > 0.f ? m1 + log2f(l1) : -INFINITY;
        }
    }
}

// The workspace after the decode attention's own: the rows' entries, the
// slots' log-sum-exps and outputs.
struct PrefixPlan {
    size_t rows, lse, part, total;
    int tile_rows, target;
};

bool prefix_plan(const mi_dims* dims, int32_t num_prefixes, int32_t max_prefix_blocks, PrefixPlan* s) {
    if (check_paged_dims(dims) != MI_OK || num_prefixes < 0 || num_prefixes > 65535 || max_prefix_blocks < 1 ||
        (long long)max_prefix_blocks * kBlock > 0x7FFFFFFFLL)
        return false;
    const size_t base = mi_paged_decode_workspace_bytes(dims);
    const int sms = sm_count();
    if (base == 0 || sms <= 0) return false;
    const mi_dims& D = *dims;
    const int G = D.Hq / D.Hkv;
    s->tile_rows = kTileRows / G * G;
    s->target = 2 * sms;
    // splits are at least total / target blocks long, so the items are at
    // most `target` and one more for every (tile, head)
    const long long per = s->tile_rows / G;
    const long long slots = s->target + (long long)D.Hkv * ((D.B + per - 1) / per + num_prefixes);
    if (slots * s->tile_rows > 0x7FFFFFFFLL) return false;
    s->rows = (base + 255) / 256 * 256;
    s->lse = s->rows + ((size_t)D.B * 16 + 255) / 256 * 256;
    s->part = s->lse + ((size_t)slots * s->tile_rows * 4 + 255) / 256 * 256;
    s->total = s->part + (size_t)slots * s->tile_rows * D.head_dim * 4;
    return true;
}

template <int HD>
bool prepare_prefix(int smem) {
    static std::mutex mu;
    static CUcontext done[256] = {};
    return raise_smem(reinterpret_cast<const void*>(prefix_kernel<HD>), smem, done, mu);
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_paged_prefix_workspace_bytes(const mi_dims* dims, int32_t num_prefixes,
                                                  int32_t max_prefix_blocks) {
    mi::PrefixPlan s;
    return mi::prefix_plan(dims, num_prefixes, max_prefix_blocks, &s) ? s.total : 0;
}

extern "C" mi_status mi_paged_decode_attention_prefix(const mi_dims* dims, int32_t num_prefixes,
                                                      int32_t max_prefix_blocks, const void* q, const void* k_cache,
                                                      const void* v_cache, const int32_t* prefix_tables,
                                                      const int32_t* prefix_lens, const int32_t* group_start,
                                                      const int32_t* block_tables, const int32_t* context_lens,
                                                      float scale, void* out, void* workspace, size_t workspace_bytes,
                                                      int32_t* dev_err, mi_stream_t stream) {
    using namespace mi;
    const mi_status ds = check_paged_dims(dims);
    if (ds != MI_OK) return ds;
    const mi_dims D = *dims;
    if (num_prefixes < 0 || num_prefixes > 65535 || max_prefix_blocks < 1 ||
        (long long)max_prefix_blocks * kBlock > 0x7FFFFFFFLL || !std::isfinite(scale))
        return MI_ERR_INVALID_ARG;
    if (D.B == 0) return MI_OK;
    if (!q || !k_cache || !v_cache || !group_start || !block_tables || !context_lens || !out || !workspace ||
        (num_prefixes > 0 && (!prefix_tables || !prefix_lens)))
        return MI_ERR_INVALID_ARG;
    if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
        !aligned_to(workspace, 16))
        return MI_ERR_INVALID_ARG;
    PrefixPlan s;
    if (!prefix_plan(dims, num_prefixes, max_prefix_blocks, &s)) return MI_ERR_CUDA;
    if (workspace_bytes < s.total) return MI_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PrefixParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k_cache);
    p.v = static_cast<const uint16_t*>(v_cache);
    p.tables = prefix_tables;
    p.lens = prefix_lens;
    p.starts = group_start;
    p.rows = reinterpret_cast<int4*>(ws + s.rows);
    p.part = reinterpret_cast<float*>(ws + s.part);
    p.part_lse = reinterpret_cast<float*>(ws + s.lse);
    p.dev_err = dev_err;
    p.P = num_prefixes;
    p.B = D.B;
    p.Hq = D.Hq;
    p.Hkv = D.Hkv;
    p.G = D.Hq / D.Hkv;
    p.num_blocks = D.num_blocks;
    p.mbps = max_prefix_blocks;
    p.tile_rows = s.tile_rows;
    p.target = s.target;
    p.sl2 = scale * 1.4426950408889634f;
    const int HD = D.head_dim, smem = 3 * kTileRows * (HD == 128 ? kPitch<128> : kPitch<64>);
    if (!(HD == 128 ? prepare_prefix<128>(smem) : prepare_prefix<64>(smem))) return MI_ERR_CUDA;
    const cudaError_t e = launch_pdl(HD == 128 ? prefix_kernel<128> : prefix_kernel<64>, s.target, kTileThreads, smem,
                                     (cudaStream_t)stream, p);
    if (e != cudaSuccess) return MI_ERR_CUDA;
    DecodeExt ext;
    ext.kind = kExtPrefix;
    ext.rows = p.rows;
    ext.part = p.part;
    ext.part_lse = p.part_lse;
    ext.slot_rows = s.tile_rows;
    return decode_attention_ext(dims, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale, out,
                                workspace, s.rows, dev_err, stream, false, ext);
}
