// What the decode attention file offers to the entry points built on it: the
// scored step's extension of the attention kernel, and the requests' own
// tokens of the shared-prefix step.
#pragma once

#include <cuda_runtime.h>

#include "mi.h"
#include "prefix.cuh"

namespace mi {

enum DecodeExtKind { kExtNone = 0, kExtScored = 1 };

struct DecodeExt {
    int kind = kExtNone;
    // kExtScored: the base-2 logits of every token, logits[e][16][gp] for KV
    // block e of a head (e: the block's place in the batch's flat (request,
    // head, block) order, or block id * Hkv + head with `by_block`), gp the
    // group size rounded up to even; and each row's log2-sum-exp [B][Hq]
    float* logits = nullptr;
    float* lse = nullptr;
    int by_block = 0, gp = 0;
};

// mi_paged_decode_attention (or the e4m3 call with `fp8`) with an extension;
// `workspace` is that of mi_paged_decode_workspace_bytes.
mi_status decode_attention_ext(const mi_dims* dims, const void* q, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, const int32_t* block_tables,
                               const int32_t* context_lens, float scale, void* out, void* workspace,
                               size_t workspace_bytes, int32_t* dev_err, mi_stream_t stream, bool fp8,
                               const DecodeExt& ext);

// Attention over the requests' own tokens in pieces: request b's piece c of KV
// head h is piece rows[b].x + h * rows[b].y + c, whose G rows of normalised
// output are part[piece][G][HD] and their log2-sum-exps lse[piece][G]; at most
// `most` + B * Hkv pieces. `prefix`, `prefix_mbps`: the prefix part that runs
// at the same time.
struct TailWork {
    int2* rows = nullptr;  // [B] {first piece, pieces per head}
    float* part = nullptr;
    float* lse = nullptr;
    long long most = 0;
    PrefixWork prefix;
    int prefix_mbps = 0;
};
constexpr int kTailLeast = 4;  // blocks: a shorter piece does not pay for its result
mi_status prefix_tail(const mi_dims* dims, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* context_lens, float scale, const TailWork& work,
                      int32_t* dev_err, mi_stream_t stream);

}  // namespace mi
