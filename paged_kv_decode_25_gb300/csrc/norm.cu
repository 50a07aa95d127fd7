// mi_paged_kv_append_norm: the append of mi_paged_kv_append for models that
// norm every query and key head before the rotation (Qwen3). For a head's d
// values x and its weights w
//   r = 1 / sqrt(sum x^2 / d + eps),  y = x r w,
//   out[i] = y[i] c - y[i + d/2] s,  out[i + d/2] = y[i + d/2] c + y[i] s
// in fp32, rounded once (to bf16, or to e4m3 of out / scale); v goes along. As
// separate steps the norm alone would move q and k twice more.
//
// Bound by the bytes of q, k, v in and out; about eight instructions a value.
// A head is HD / 16 lanes, each holding eight values of its lower half and the
// eight they are rotated with, so the sum of squares is two or three shuffles
// and the rotation none; a warp has 4 (head_dim 128) or 8 heads at once. A row's
// groups of heads go to as many warps as fill the device: all of a row's to one
// (its cosines, sines and weights are then read once) where there are many rows.
//
// Measured: 12,821 tokens (32/8 heads of 128, bf16, one projection's rows) 52 us, 6.2 TB/s,
// 91 % of a copy's rate; 5,000 tokens into e4m3 (28/4) 20.2 us, 4.4 TB/s: 1.6 waves of
// blocks, fp32 arithmetic value by value, 12 bytes of spill (16.6 where inputs are in
// L2; 18.3 with a product for a quotient); a step of 64 tokens 2.3 us on the
// device. Five blocks an SM (96 registers), four groups' loads in flight: 55 us with four
// blocks, 58 with two groups. A row in one warp from 16 warps an SM on: parts of rows
// read cosines and weights again (5,000 tokens: 22.5 us in bf16, 23.7 from 40 on).
#include "batch.cuh"
#include "common.cuh"

namespace mi {
namespace {

constexpr int kNormWarps = 4;
constexpr int kNormBatch = 4;  // groups of heads whose loads a warp has in flight

struct NormParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    long long q_stride, k_stride, v_stride;  // elements between rows
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    const int32_t* positions;
    const int32_t* slot_mapping;
    const float2* rope;  // [max_pos][d/2] (cos, sin)
    uint16_t* q_out;
    uint8_t* k_cache;
    uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    int32_t* dev_err;
    float eps;
    int B, Hq, Hkv, num_blocks, max_pos;
    int per, parts;  // groups of a row that one warp takes, warps of a row
};

__device__ __forceinline__ bool norm_scale_ok(float s) { return s > 0.f && s <= 3.0e38f; }

// Quotients by one head's scale in IEEE single precision. With r = 1 / s correctly
// rounded and q within one ulp of y / s, q plus its exact remainder times r, rounded
// once, is the correctly rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990); y r
// may be 1.5 ulp off, so it is corrected twice. Remainders are exact and nothing
// overflows for scales between 2^-60 and 2^60 and quotients below 1,024; larger ones
// saturate whatever their last bit, and where y is too small for an exact remainder the
// quotient is far below half of e4m3's smallest value. Other scales divide, out of line.
// (8,000 tokens, 32/8 heads: 37 us; dividing always 39; with a mere product 33.)
struct Divisor {
    float s, r;
    bool plain;
    __device__ __forceinline__ explicit Divisor(float scale) : s(scale) {
        r = __fdiv_rn(1.f, scale);
        plain = scale >= 0x1p-60f && scale <= 0x1p60f;
    }
    __device__ __forceinline__ float corrected(float y) const {
        const float q = y * r, p = fmaf(fmaf(-q, s, y), r, q);
        const float z = fmaf(fmaf(-p, s, y), r, p);
        return fabsf(q) < 1024.f ? copysignf(z, q) : q;  // (a zero's remainder loses its sign)
    }
};

__device__ __noinline__ float divided(float y, float s) { return __fdiv_rn(y, s); }

// Eight values / scale, then e4m3.
__device__ __forceinline__ uint2 e4m3x8(const float (&y)[8], const Divisor& by) {
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = by.corrected(y[j]);
    if (!by.plain) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = divided(y[j], by.s);
    }
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = f32x2_to_e4m3x2(z[2 * j], z[2 * j + 1]);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(u[j]);
        x[2 * j + 1] = bf16_hi(u[j]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                      pack_bf16x2(y[6], y[7]));
}

template <int HD, bool FP8>
__global__ void __launch_bounds__(kNormWarps * 32, 5) norm_append_kernel(const NormParams a) {
    constexpr int kLanes = HD / 16;      // of a head
    constexpr int kHeads = 32 / kLanes;  // of a group
    constexpr int kChunks = HD / 8;      // 16-byte pieces of a v head
    constexpr int kEB = FP8 ? 1 : 2;
    // inputs may come from the kernel just before this one in the stream
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
    const long long row = item / a.parts;
    if (row >= a.B) return;
    const int g0 = (int)(item - row * a.parts) * a.per;
    const int rot = (a.Hq + a.Hkv + kHeads - 1) / kHeads, all = rot + (a.Hkv * kChunks + 31) / 32;
    const int g1 = min(all, g0 + a.per);
    const int pos = __ldg(a.positions + row), slot = __ldg(a.slot_mapping + row);
    if (pos < 0 || pos >= a.max_pos) {
        if (lane == 0 && g0 == 0) raise_err(a.dev_err, MI_DEVERR_BAD_POS);
        return;
    }
    const bool stored = slot >= 0 && slot < a.num_blocks * kBlock;
    if (!stored && lane == 0 && g0 == 0) raise_err(a.dev_err, MI_DEVERR_BAD_SLOT);
    // row of KV head 0 in the caches; head h's is h * 16 rows on
    const long long cell = stored ? (long long)(slot / kBlock) * a.Hkv * kBlock + slot % kBlock : 0;

    if (g0 < rot) {
        const int sub = lane / kLanes, i0 = 8 * (lane % kLanes);
        const uint4 wq_lo = __ldg(reinterpret_cast<const uint4*>(a.q_weight + i0));
        const uint4 wq_hi = __ldg(reinterpret_cast<const uint4*>(a.q_weight + i0 + HD / 2));
        const uint4 wk_lo = __ldg(reinterpret_cast<const uint4*>(a.k_weight + i0));
        const uint4 wk_hi = __ldg(reinterpret_cast<const uint4*>(a.k_weight + i0 + HD / 2));
        float c[8], s[8];
        const float4* cs = reinterpret_cast<const float4*>(a.rope + (long long)pos * (HD / 2) + i0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 t = __ldg(cs + j);
            c[2 * j] = t.x;
            s[2 * j] = t.y;
            c[2 * j + 1] = t.z;
            s[2 * j + 1] = t.w;
        }
        const uint16_t* q = a.q + row * a.q_stride + i0;
        const uint16_t* k = a.k + row * a.k_stride + i0;
        const int end = min(g1, rot);
        for (int g = g0; g < end; g += kNormBatch) {
            uint4 lo[kNormBatch], hi[kNormBatch];
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                const int head = (g + u) * kHeads + sub;
                lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
                if (g + u < end && head < a.Hq + a.Hkv) {
                    const uint16_t* x = head < a.Hq ? q + (long long)head * HD : k + (long long)(head - a.Hq) * HD;
                    lo[u] = *reinterpret_cast<const uint4*>(x);
                    hi[u] = *reinterpret_cast<const uint4*>(x + HD / 2);
                }
            }
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                if (g + u >= end) break;
                const int head = (g + u) * kHeads + sub;
                const bool is_q = head < a.Hq;
                float x[8], y[8], sum = 0.f;
                unpack8(lo[u], x);
                unpack8(hi[u], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], fmaf(y[j], y[j], sum));
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float r = rsqrtf(fmaf(sum, 1.f / HD, a.eps));
                float w[8], z[8];
                unpack8(is_q ? wq_lo : wk_lo, w);
                unpack8(is_q ? wq_hi : wk_hi, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = x[j] * r * w[j], t = y[j] * r * z[j];
                    x[j] = p * c[j] - t * s[j];
                    y[j] = t * c[j] + p * s[j];
                }
                if (is_q) {
                    uint16_t* dst = a.q_out + (row * a.Hq + head) * HD + i0;
                    *reinterpret_cast<uint4*>(dst) = pack8(x);
                    *reinterpret_cast<uint4*>(dst + HD / 2) = pack8(y);
                } else if (stored && head < a.Hq + a.Hkv) {
                    const int h = head - a.Hq;
                    uint8_t* dst = a.k_cache + ((cell + (long long)h * kBlock) * HD + i0) * kEB;
                    if constexpr (FP8) {
                        const float ks = __ldg(a.k_scale + h);
                        if (norm_scale_ok(ks)) {
                            const Divisor by(ks);
                            *reinterpret_cast<uint2*>(dst) = e4m3x8(x, by);
                            *reinterpret_cast<uint2*>(dst + HD / 2) = e4m3x8(y, by);
                        } else if (i0 == 0) {
                            raise_err(a.dev_err, MI_DEVERR_BAD_SCALE);
                        }
                    } else {
                        *reinterpret_cast<uint4*>(dst) = pack8(x);
                        *reinterpret_cast<uint4*>(dst + HD) = pack8(y);
                    }
                }
            }
        }
    }
    if (!stored) return;
    const uint16_t* v = a.v + row * a.v_stride;
    for (int g = max(g0, rot) - rot; g < g1 - rot; g += kNormBatch) {
        uint4 x[kNormBatch];
#pragma unroll
        for (int u = 0; u < kNormBatch; ++u) {
            const int i = (g + u) * 32 + lane;
            if (g + u < g1 - rot && i < a.Hkv * kChunks) x[u] = *reinterpret_cast<const uint4*>(v + 8LL * i);
        }
#pragma unroll
        for (int u = 0; u < kNormBatch; ++u) {
            const int i = (g + u) * 32 + lane;
            if (g + u < g1 - rot && i < a.Hkv * kChunks) {
                const int h = i / kChunks, ch = i % kChunks;
                uint8_t* dst = a.v_cache + ((cell + (long long)h * kBlock) * HD + 8 * ch) * kEB;
                if constexpr (FP8) {
                    const float vs = __ldg(a.v_scale + h);
                    if (norm_scale_ok(vs)) {
                        float y[8];
                        unpack8(x[u], y);
                        *reinterpret_cast<uint2*>(dst) = e4m3x8(y, Divisor(vs));
                    } else if (ch == 0) {
                        raise_err(a.dev_err, MI_DEVERR_BAD_SCALE);
                    }
                } else {
                    *reinterpret_cast<uint4*>(dst) = x[u];
                }
            }
        }
    }
}

mi_status append_norm(const mi_dims* dims, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                      const int32_t* positions, const int32_t* slot_mapping, const float* rope_cos_sin, int32_t max_pos,
                      void* q_out, void* k_cache, void* v_cache, const float* k_scale, const float* v_scale, bool fp8,
                      int32_t* dev_err, mi_stream_t stream) {
    if (!dims) return MI_ERR_INVALID_ARG;
    const mi_dims D = *dims;
    if (D.B < 0 || D.B > (1 << 24) || D.Hq < 1 || D.Hkv < 1 || D.num_blocks < 1 || max_pos < 1)
        return MI_ERR_INVALID_ARG;
    if (D.block_size != kBlock || (D.head_dim != 64 && D.head_dim != 128) || D.Hq % D.Hkv != 0)
        return MI_ERR_UNSUPPORTED;
    if ((long long)D.num_blocks * kBlock > 0x7FFFFFFFLL) return MI_ERR_INVALID_ARG;
    const long long HD = D.head_dim, q_row = D.Hq * HD, kv_row = D.Hkv * HD;
    if ((D.Hq + 2LL * D.Hkv) * HD > 0x7FFFFFFFLL) return MI_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps <= 3.0e38f)) return MI_ERR_INVALID_ARG;
    if (D.B == 0) return MI_OK;
    if (!q || !k || !v || !q_weight || !k_weight || !positions || !slot_mapping || !rope_cos_sin || !q_out || !k_cache ||
        !v_cache)
        return MI_ERR_INVALID_ARG;
    if (fp8 && (!k_scale || !v_scale)) return MI_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, q_weight, k_weight, (const void*)rope_cos_sin, (const void*)q_out,
                          (const void*)k_cache, (const void*)v_cache})
        if (!aligned_to(p, 16)) return MI_ERR_INVALID_ARG;
    const int64_t strides[3] = {q_stride, k_stride, v_stride};
    const long long rows[3] = {q_row, kv_row, kv_row};
    const void* from[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] % 8 != 0 || strides[i] < rows[i] || strides[i] > (1LL << 36)) return MI_ERR_INVALID_ARG;
        // q_out is either q itself or apart from what is read
        if (i == 0 && q == q_out && (q_stride == q_row || D.B == 1)) continue;
        if (overlaps(from[i], (size_t)(((D.B - 1LL) * strides[i] + rows[i]) * 2), q_out, (size_t)(D.B * q_row * 2)))
            return MI_ERR_INVALID_ARG;
    }
    NormParams a;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = static_cast<const uint16_t*>(q_weight);
    a.k_weight = static_cast<const uint16_t*>(k_weight);
    a.positions = positions;
    a.slot_mapping = slot_mapping;
    a.rope = reinterpret_cast<const float2*>(rope_cos_sin);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.dev_err = dev_err;
    a.eps = eps;
    a.B = D.B;
    a.Hq = D.Hq;
    a.Hkv = D.Hkv;
    a.num_blocks = D.num_blocks;
    a.max_pos = max_pos;
    const int heads = 512 / D.head_dim;
    const long long groups = (D.Hq + (long long)D.Hkv + heads - 1) / heads + (kv_row / 8 + 31) / 32;
    const int sms = sm_count();
    if (sms <= 0) return MI_ERR_CUDA;
    // warps of a row: enough for 16 to an SM, at most one per group
    const long long want = (16LL * sms + D.B - 1) / D.B;
    const long long parts = want < groups ? want : groups;
    a.per = (int)((groups + parts - 1) / parts);
    a.parts = (int)((groups + a.per - 1) / a.per);
    const long long grid = ((long long)D.B * a.parts + kNormWarps - 1) / kNormWarps;
    if (grid > 0x7FFFFFFFLL) return MI_ERR_INVALID_ARG;
    const cudaStream_t st = (cudaStream_t)stream;
    const auto fn = D.head_dim == 64 ? (fp8 ? norm_append_kernel<64, true> : norm_append_kernel<64, false>)
                                     : (fp8 ? norm_append_kernel<128, true> : norm_append_kernel<128, false>);
    return launch_pdl(fn, (int)grid, kNormWarps * 32, 0, st, a) == cudaSuccess ? MI_OK : MI_ERR_CUDA;
}

}  // namespace
}  // namespace mi

extern "C" mi_status mi_paged_kv_append_norm(const mi_dims* dims, const void* q, int64_t q_stride, const void* k,
                                             int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                                             const void* k_weight, float eps, const int32_t* positions,
                                             const int32_t* slot_mapping, const float* rope_cos_sin, int32_t max_pos,
                                             void* q_out, void* k_cache, void* v_cache, int32_t* dev_err,
                                             mi_stream_t stream) {
    return mi::append_norm(dims, q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, positions, slot_mapping,
                           rope_cos_sin, max_pos, q_out, k_cache, v_cache, nullptr, nullptr, false, dev_err, stream);
}

extern "C" mi_status mi_paged_kv_append_norm_fp8(const mi_dims* dims, const void* q, int64_t q_stride, const void* k,
                                                 int64_t k_stride, const void* v, int64_t v_stride,
                                                 const void* q_weight, const void* k_weight, float eps,
                                                 const int32_t* positions, const int32_t* slot_mapping,
                                                 const float* rope_cos_sin, int32_t max_pos, void* q_out, void* k_cache,
                                                 void* v_cache, const float* k_scale, const float* v_scale,
                                                 int32_t* dev_err, mi_stream_t stream) {
    return mi::append_norm(dims, q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, positions, slot_mapping,
                           rope_cos_sin, max_pos, q_out, k_cache, v_cache, k_scale, v_scale, true, dev_err, stream);
}
