// mi_paged_decode_attention_scored: decode attention that also keeps, for every
// cached token and KV head, the attention weight the token has received.
//
//   score[b][h][t] (+)= sum over the G query heads j of h of
//                       2^(x_jt - lse_j),   x the base-2 logits
//
// A weight needs its row's final log-sum-exp, so the attention kernel (the
// decode kernel of decode.cu) writes each logit as it streams K and V, and
// this pass turns them into weights once every row is finished. The logits
// are 4 G bytes of a token's 512 (bf16, head_dim 128) per KV head; the
// alternative, K read again, would be 256.
#include "batch.cuh"
#include "decode.cuh"

namespace mi {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 1024;  // of one (request, head) per work item

struct ScoreParams {
    const int32_t* tables;         // [B][mbps]
    const int32_t* lens;           // [B]
    const float* logits;           // [blocks][16][GP], see DecodeExt
    const float* lse;              // [B][Hq]
    float* scores;                 // [num_blocks][Hkv][16]
    int B, Hq, Hkv, G, num_blocks, mbps, by_block, fresh;
};

// GP: floats of a token's logits. A thread takes four consecutive tokens of a
// block, so that all its loads (4 GP floats of logits, a table entry, four
// scores) are wide and, but for the scores, independent. Latency bounds it: 11
// us for the 23 MB of logits and 12 MB of scores of 64 requests of 512 to 8,192
// tokens, all of it in L2.
template <int GP>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const ScoreParams p) {
    __shared__ long long sums[flat_words(kScoreThreads)], bsums[flat_words(kScoreThreads)];
    // the plan and the first item's table entries need nothing of the attention,
    // which had waited for all before it
    bool waited = false;
    auto wait = [&]() {
        if (waited) return;
        pdl_wait();
        pdl_trigger();
        waited = true;
    };
    auto tokens = [&](int b) { return min(max(__ldg(p.lens + b), 0), p.mbps * kBlock); };
    // work items are 64 blocks of one (request, head); the logits of the
    // flat order lie in blocks of (request, head) laid end to end
    constexpr int kItemBlocks = kScoreTokens / kBlock;
    auto items = [&](int b) { return (long long)p.Hkv * ((tokens(b) + kScoreTokens - 1) / kScoreTokens); };
    auto blocks = [&](int b) { return (long long)p.Hkv * ((tokens(b) + kBlock - 1) / kBlock); };
    const long long total = flat_scan(p.B, items, sums);
    if (!p.by_block) flat_scan(p.B, blocks, bsums);
    for (long long x = blockIdx.x; x < total; x += gridDim.x) {
        long long first;
        const int b = flat_find(p.B, items, sums, x, first);
        const int n = tokens(b), nblk = (n + kBlock - 1) / kBlock, per = (n + kScoreTokens - 1) / kScoreTokens;
        const int o = (int)(x - first), h = o / per, j0 = (o % per) * kItemBlocks;
        const long long e0 = p.by_block ? 0 : flat_before(p.B, blocks, bsums, b) + (long long)h * nblk;
        const int j = j0 + threadIdx.x / 4, i0 = threadIdx.x % 4 * 4, t0 = j * kBlock + i0;
        if (t0 >= n) continue;
        const int blk = __ldg(p.tables + (long long)b * p.mbps + j);
        const bool in = blk >= 0 && blk < p.num_blocks;  // (else reported by the attention)
        if (!in && p.by_block) continue;
        wait();
        const long long e = p.by_block ? (long long)blk * p.Hkv + h : e0 + j;
        const float* lg = p.logits + (e * kBlock + i0) * GP;
        float l[4 * GP], lse[GP];
#pragma unroll
        for (int c = 0; c < GP; ++c) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(lg) + c);
            l[4 * c] = v.x;
            l[4 * c + 1] = v.y;
            l[4 * c + 2] = v.z;
            l[4 * c + 3] = v.w;
        }
#pragma unroll
        for (int g = 0; g < GP; ++g)
            lse[g] = g < p.G ? __ldcg(p.lse + (long long)b * p.Hq + (long long)h * p.G + g) : INFINITY;
        if (!in) continue;
        float4* at = reinterpret_cast<float4*>(p.scores + ((long long)blk * p.Hkv + h) * kBlock + i0);
        const bool whole = p.fresh && t0 + 4 <= n;
        const float4 old = whole ? make_float4(0.f, 0.f, 0.f, 0.f) : *at;
        float w[4], was[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < GP; ++g)
                if (g < p.G) v += exp2f(l[c * GP + g] - lse[g]);
            const int t = t0 + c;
            w[c] = t >= n ? was[c] : p.fresh || t == n - 1 ? v : was[c] + v;
        }
        *at = make_float4(w[0], w[1], w[2], w[3]);
    }
    wait();  // (whoever waits for this launch has the attention too)
}

// The workspace after the decode attention's own: each row's log-sum-exp,
// then the logits.
struct ScoredPlan {
    size_t lse, logits, total;
    int gp, by_block;
};

bool scored_plan(const mi_dims* dims, ScoredPlan* s) {
    if (check_paged_dims(dims) != MI_OK) return false;
    const size_t base = mi_paged_decode_workspace_bytes(dims);
    if (base == 0) return false;
    const mi_dims& D = *dims;
    s->gp = (D.Hq / D.Hkv + 1) / 2 * 2;
    // logits by the batch's flat order of blocks, or by the cache's, whichever
    // has fewer places
    const long long flat = (long long)D.B * D.max_blocks_per_seq;
    s->by_block = flat > D.num_blocks;
    const size_t places = (size_t)(s->by_block ? D.num_blocks : flat) * D.Hkv;
    s->lse = (base + 255) / 256 * 256;
    s->logits = s->lse + ((size_t)D.B * D.Hq * 4 + 255) / 256 * 256;
    s->total = s->logits + places * kBlock * s->gp * 4;
    return true;
}

mi_status scored(const mi_dims* dims, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                 const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, float scale,
                 int32_t fresh, void* out, float* scores, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                 mi_stream_t stream, bool fp8) {
    const mi_status ds = check_paged_dims(dims);
    if (ds != MI_OK) return ds;
    const mi_dims D = *dims;
    if (D.B == 0) return MI_OK;
    if (!scores || !workspace || !block_tables || !context_lens) return MI_ERR_INVALID_ARG;
    if (!aligned_to(scores, 16) || !aligned_to(workspace, 16)) return MI_ERR_INVALID_ARG;
    ScoredPlan s;
    if (!scored_plan(dims, &s)) return MI_ERR_CUDA;
    if (workspace_bytes < s.total) return MI_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return MI_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    DecodeExt ext;
    ext.kind = kExtScored;
    ext.logits = reinterpret_cast<float*>(ws + s.logits);
    ext.lse = reinterpret_cast<float*>(ws + s.lse);
    ext.by_block = s.by_block;
    ext.gp = s.gp;
    const mi_status st = decode_attention_ext(dims, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                              scale, out, workspace, s.lse, dev_err, stream, fp8, ext);
    if (st != MI_OK) return st;
    ScoreParams p;
    p.tables = block_tables;
    p.lens = context_lens;
    p.logits = ext.logits;
    p.lse = ext.lse;
    p.scores = scores;
    p.B = D.B;
    p.Hq = D.Hq;
    p.Hkv = D.Hkv;
    p.G = D.Hq / D.Hkv;
    p.num_blocks = D.num_blocks;
    p.mbps = D.max_blocks_per_seq;
    p.by_block = s.by_block;
    p.fresh = fresh != 0;
    const long long most = (long long)D.B * D.Hkv * (((long long)D.max_blocks_per_seq * kBlock + kScoreTokens - 1) / kScoreTokens);
    const int grid = (int)(most < 8LL * sms ? most : 8LL * sms);
    void (*const kernel[4])(ScoreParams) = {score_kernel<2>, score_kernel<4>, score_kernel<6>, score_kernel<8>};
    return launch_pdl(kernel[s.gp / 2 - 1], grid, kScoreThreads, 0, (cudaStream_t)stream, p) == cudaSuccess ? MI_OK
                                                                                                           : MI_ERR_CUDA;
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_paged_scored_workspace_bytes(const mi_dims* dims) {
    mi::ScoredPlan s;
    return mi::scored_plan(dims, &s) ? s.total : 0;
}

extern "C" mi_status mi_paged_decode_attention_scored(const mi_dims* dims, const void* q, const void* k_cache,
                                                      const void* v_cache, const int32_t* block_tables,
                                                      const int32_t* context_lens, float scale, int32_t fresh,
                                                      void* out, float* scores, void* workspace,
                                                      size_t workspace_bytes, int32_t* dev_err, mi_stream_t stream) {
    return mi::scored(dims, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale, fresh, out,
                      scores, workspace, workspace_bytes, dev_err, stream, false);
}

extern "C" mi_status mi_paged_decode_attention_scored_fp8(const mi_dims* dims, const void* q, const void* k_cache,
                                                          const void* v_cache, const float* k_scale,
                                                          const float* v_scale, const int32_t* block_tables,
                                                          const int32_t* context_lens, float scale, int32_t fresh,
                                                          void* out, float* scores, void* workspace,
                                                          size_t workspace_bytes, int32_t* dev_err,
                                                          mi_stream_t stream) {
    return mi::scored(dims, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, fresh, out,
                      scores, workspace, workspace_bytes, dev_err, stream, true);
}
