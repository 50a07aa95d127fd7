// mi_paged_decode_attention_prefix: one decode step of a batch whose requests
// share prefixes, each prefix's keys and values read once for all of them.
//
// Request b of group g attends to the prefix's tokens followed by its own.
// The softmax over the two parts is put together from their (output,
// log-sum-exp) pairs, so the parts are computed apart:
//   * prefix_partials (prefill.cu): the group's queries against the prefix on
//     the fifth-generation tensor cores, as one tall matrix of (request, head)
//     rows per KV head: a staged K / V tile serves up to 256 of them;
//   * prefix_tail (decode.cu): the requests' own blocks, a warp per piece, at
//     the same time on the SMs that the first part leaves;
//   * prefix_merge_kernel puts each row together from the two.
//
// The rows of (group, KV head) are cut into tiles of whole requests, the
// prefix's blocks into equal splits; a (group, tile, split, head) is a work
// item of one block and writes one slot of partial results (prefix.cuh).
#include <cmath>

#include "batch.cuh"
#include "decode.cuh"
#include "prefix.cuh"

namespace mi {
namespace {

constexpr int kMergeThreads = 256;

struct MergeParams {
    const int4* prefix_rows;       // [B] see PrefixWork
    const float* prefix_part;
    const float* prefix_lse;
    const int2* tail_rows;         // [B] see TailWork
    const float* tail_part;
    const float* tail_lse;
    uint16_t* out;                 // [B][Hq][HD]
    int B, Hq, Hkv, G, slot_rows;
};

// out = sum 2^(lse_i - M) o_i / sum 2^(lse_i - M) over a row's partial results,
// the prefix's splits first, in order. HD / 4 lanes hold a row: each fetches
// the log-sum-exps of every (HD / 4)-th part, so that the weights cost one
// round of loads, and the outputs are then independent of one another.
template <int HD>
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const MergeParams p) {
    constexpr int L = HD / 4, kRows = kMergeThreads / L;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sub = threadIdx.x & (L - 1), src = lane & ~(L - 1);
    const unsigned lanes = L == 32 ? 0xffffffffu : 0xffffu << src;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / L;
    if (row >= (long long)p.B * p.Hq) return;
    const int b = (int)(row / p.Hq), j = (int)(row % p.Hq), h = j / p.G, g = j % p.G;
    const int4 at = __ldcg(p.prefix_rows + b);
    const int2 own = __ldcg(p.tail_rows + b);
    const int parts = at.y + own.y;
    // where part i's row lies, in rows of its array
    auto place = [&](int i) {
        return i < at.y ? (long long)(at.x + i * p.Hkv + h) * p.slot_rows + at.z + g
                        : (long long)(own.x + h * own.y + (i - at.y)) * p.G + g;
    };
    float M = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += L) {
        const int cnt = min(parts - i0, L);
        float mine = -INFINITY;
        if (sub < cnt) mine = __ldcg((i0 + sub < at.y ? p.prefix_lse : p.tail_lse) + place(i0 + sub));
        float top = mine;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, o));
        top = fmaxf(top, M);
        if (top == -INFINITY) continue;
        const float old = exp2f(M - top), w = exp2f(mine - top);
        M = top;
        float ws = w;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ws += __shfl_xor_sync(lanes, ws, o);
        den = den * old + ws;
        num = make_float4(num.x * old, num.y * old, num.z * old, num.w * old);
#pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const float wk = __shfl_sync(lanes, w, src + k);
            const float4 o = __ldcg(reinterpret_cast<const float4*>((i0 + k < at.y ? p.prefix_part : p.tail_part) +
                                                                    place(i0 + k) * HD + sub * 4));
            num.x += wk * o.x;
            num.y += wk * o.y;
            num.z += wk * o.z;
            num.w += wk * o.w;
        }
    }
    const float r = den > 0.f ? 1.f / den : 0.f;
    *reinterpret_cast<uint2*>(p.out + row * HD + sub * 4) =
        make_uint2(pack_bf16x2(num.x * r, num.y * r), pack_bf16x2(num.z * r, num.w * r));
}

// The workspace: the requests' entries of both parts, the log-sum-exps and
// outputs of the prefix's slots and of the pieces.
struct PrefixSpace {
    size_t rows, tail_rows, lse, tail_lse, part, tail_part, total;
    long long slots;
    int slot_rows, sms, most;
};

bool prefix_space(const mi_dims* dims, int32_t num_prefixes, int32_t max_prefix_blocks, PrefixSpace* s) {
    if (check_paged_dims(dims) != MI_OK || num_prefixes < 0 || num_prefixes > 65535 || max_prefix_blocks < 1 ||
        max_prefix_blocks > kLongestTable)
        return false;
    const int sms = sm_count();
    if (sms <= 0) return false;
    const mi_dims& D = *dims;
    const int G = D.Hq / D.Hkv, per = prefix_tile_requests(G);
    s->sms = sms;
    s->slot_rows = per * G;
    s->slots = prefix_slots(D.B, D.Hkv, num_prefixes, per, sms);
    s->most = 32 * sms;
    const long long pieces = s->most + (long long)D.B * D.Hkv;
    if (s->slots * s->slot_rows > 0x7FFFFFFFLL || pieces * G > 0x3FFFFFFFLL) return false;
    auto next = [](size_t at, size_t bytes) { return (at + bytes + 255) / 256 * 256; };
    s->rows = 0;
    s->tail_rows = next(s->rows, (size_t)D.B * 16);
    s->lse = next(s->tail_rows, (size_t)D.B * 8);
    s->tail_lse = next(s->lse, (size_t)s->slots * s->slot_rows * 4);
    s->part = next(s->tail_lse, (size_t)pieces * G * 4);
    s->tail_part = next(s->part, (size_t)s->slots * s->slot_rows * D.head_dim * 4);
    s->total = next(s->tail_part, (size_t)pieces * G * D.head_dim * 4);
    return true;
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_paged_prefix_workspace_bytes(const mi_dims* dims, int32_t num_prefixes,
                                                  int32_t max_prefix_blocks) {
    mi::PrefixSpace s;
    return mi::prefix_space(dims, num_prefixes, max_prefix_blocks, &s) ? s.total : 0;
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
        max_prefix_blocks > kLongestTable || !std::isfinite(scale))
        return MI_ERR_INVALID_ARG;
    if (D.B == 0) return MI_OK;
    if (!q || !k_cache || !v_cache || !group_start || !block_tables || !context_lens || !out || !workspace ||
        (num_prefixes > 0 && (!prefix_tables || !prefix_lens)))
        return MI_ERR_INVALID_ARG;
    if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
        !aligned_to(workspace, 16))
        return MI_ERR_INVALID_ARG;
    PrefixSpace s;
    if (!prefix_space(dims, num_prefixes, max_prefix_blocks, &s)) return MI_ERR_CUDA;
    if (workspace_bytes < s.total) return MI_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PrefixWork w;
    w.lens = prefix_lens;
    w.starts = group_start;
    w.rows = reinterpret_cast<int4*>(ws + s.rows);
    w.part = reinterpret_cast<float*>(ws + s.part);
    w.part_lse = reinterpret_cast<float*>(ws + s.lse);
    w.own = context_lens;
    w.own_blocks = D.max_blocks_per_seq;
    w.P = num_prefixes;
    w.B = D.B;
    w.sms = s.sms;
    mi_status st = prefix_partials(dims, max_prefix_blocks, q, k_cache, v_cache, prefix_tables, scale, w, s.slots,
                                         dev_err, stream);
    if (st != MI_OK) return st;
    TailWork t;
    t.rows = reinterpret_cast<int2*>(ws + s.tail_rows);
    t.part = reinterpret_cast<float*>(ws + s.tail_part);
    t.lse = reinterpret_cast<float*>(ws + s.tail_lse);
    t.most = s.most;
    t.prefix = w;
    t.prefix_mbps = max_prefix_blocks;
    st = prefix_tail(dims, q, k_cache, v_cache, block_tables, context_lens, scale, t, dev_err, stream);
    if (st != MI_OK) return st;
    MergeParams m;
    m.prefix_rows = w.rows;
    m.prefix_part = w.part;
    m.prefix_lse = w.part_lse;
    m.tail_rows = t.rows;
    m.tail_part = t.part;
    m.tail_lse = t.lse;
    m.out = static_cast<uint16_t*>(out);
    m.B = D.B;
    m.Hq = D.Hq;
    m.Hkv = D.Hkv;
    m.G = D.Hq / D.Hkv;
    m.slot_rows = s.slot_rows;
    const int HD = D.head_dim, per = kMergeThreads / (HD / 4);
    const long long grid = ((long long)D.B * D.Hq + per - 1) / per;
    if (grid > 0x7FFFFFFFLL) return MI_ERR_INVALID_ARG;
    return launch_pdl(HD == 128 ? prefix_merge_kernel<128> : prefix_merge_kernel<64>, (int)grid, kMergeThreads, 0,
                      (cudaStream_t)stream, m) == cudaSuccess
               ? MI_OK
               : MI_ERR_CUDA;
}
