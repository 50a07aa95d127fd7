// What the decode attention kernel does on top of plain attention for the
// entry points built on it (the scored step and the shared-prefix step).
#pragma once

#include <cuda_runtime.h>

#include "mi.h"

namespace mi {

enum DecodeExtKind { kExtNone = 0, kExtScored = 1, kExtPrefix = 2 };

struct DecodeExt {
    int kind = kExtNone;
    // kExtScored: the base-2 logits of every token, logits[e][16][gp] for KV
    // block e of a head (e: the block's place in the batch's flat (request,
    // head, block) order, or block id * Hkv + head with `by_block`), gp the
    // group size rounded up to even; and each row's log2-sum-exp [B][Hq]
    float* logits = nullptr;
    float* lse = nullptr;
    int by_block = 0, gp = 0;
    // kExtPrefix: what to merge into the rows of request b: rows[b] = {first
    // slot, splits, row in the slot, 0}; split s of KV head h is slot first +
    // s * Hkv + h, whose row i holds a normalised output part[(slot *
    // slot_rows + i) * HD ..] and its log2-sum-exp part_lse[slot * slot_rows + i]
    const int4* rows = nullptr;
    const float* part = nullptr;
    const float* part_lse = nullptr;
    int slot_rows = 0;
};

// mi_paged_decode_attention (or the e4m3 call with `fp8`) with an extension;
// `workspace` is that of mi_paged_decode_workspace_bytes.
mi_status decode_attention_ext(const mi_dims* dims, const void* q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* block_tables,
                               const int32_t* context_lens, float scale, void* out, void* workspace,
                               size_t workspace_bytes, int32_t* dev_err, mi_stream_t stream, bool fp8,
                               const DecodeExt& ext);

}  // namespace mi
