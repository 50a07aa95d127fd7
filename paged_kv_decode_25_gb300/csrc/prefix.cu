// mi_paged_decode_attention_prefix: one decode step of a batch whose requests
// share prefixes, each prefix's keys and values read once for all of them.
//
// Request b of group g attends to the prefix's tokens followed by its own.
// The softmax over the two parts is put together from their (output,
// log-sum-exp) pairs, so the parts are computed apart:
//   * prefix_partials (prefill.cu): the group's queries against the prefix on
//     the fifth-generation tensor cores, as one tall matrix of (request, head)
//     rows per KV head: a staged K / V tile serves up to 256 of them;
//   * the decode kernel (decode.cu) over the requests' own blocks, which
//     merges the prefix's partial results into each row as it finishes it.
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

// The workspace after the decode attention's own: the rows' entries, the
// slots' log-sum-exps and outputs.
struct PrefixSpace {
    size_t rows, lse, part, total;
    long long slots;
    int slot_rows, sms;
};

bool prefix_space(const mi_dims* dims, int32_t num_prefixes, int32_t max_prefix_blocks, PrefixSpace* s) {
    if (check_paged_dims(dims) != MI_OK || num_prefixes < 0 || num_prefixes > 65535 || max_prefix_blocks < 1 ||
        (long long)max_prefix_blocks * kBlock > 0x7FFFFFFFLL)
        return false;
    const size_t base = mi_paged_decode_workspace_bytes(dims);
    const int sms = sm_count();
    if (base == 0 || sms <= 0) return false;
    const mi_dims& D = *dims;
    const int G = D.Hq / D.Hkv, per = prefix_tile_requests(G);
    s->sms = sms;
    s->slot_rows = per * G;
    s->slots = prefix_slots(D.B, D.Hkv, num_prefixes, per, sms);
    if (s->slots * s->slot_rows > 0x7FFFFFFFLL) return false;
    s->rows = (base + 255) / 256 * 256;
    s->lse = s->rows + ((size_t)D.B * 16 + 255) / 256 * 256;
    s->part = s->lse + ((size_t)s->slots * s->slot_rows * 4 + 255) / 256 * 256;
    s->total = s->part + (size_t)s->slots * s->slot_rows * D.head_dim * 4;
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
        (long long)max_prefix_blocks * kBlock > 0x7FFFFFFFLL || !std::isfinite(scale))
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
    w.P = num_prefixes;
    w.B = D.B;
    w.sms = s.sms;
    const mi_status st = prefix_partials(dims, max_prefix_blocks, q, k_cache, v_cache, prefix_tables, scale, w, s.slots,
                                         dev_err, stream);
    if (st != MI_OK) return st;
    DecodeExt ext;
    ext.kind = kExtPrefix;
    ext.rows = w.rows;
    ext.part = w.part;
    ext.part_lse = w.part_lse;
    ext.slot_rows = s.slot_rows;
    return decode_attention_ext(dims, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, scale, out,
                                workspace, s.rows, dev_err, stream, false, ext);
}
