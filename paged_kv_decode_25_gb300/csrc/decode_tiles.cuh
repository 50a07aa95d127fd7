// The tiles of decode attention: what one warp computes over a staged block of 16
// tokens, its (maximum, sum, output) state kept in registers. bf16, e4m3 and INT8
// caches; used by the decode attention kernels. `Params` has q, Hq, G, sl2 and the
// scales; `seen(t)` says whether token t of the block takes part.
#pragma once

#include "common.cuh"
#include "decode.cuh"
#include "tma.cuh"

namespace mi {

constexpr int kMaxG = 8;
constexpr float kNegInf = -INFINITY;

enum { kVarMma = 1, kVarFma = 2, kVarFp8 = 3, kVarInt8 = 4 };

// Bytes of one cache element: bf16, or one byte for the e4m3 and INT8 variants.
__host__ __device__ constexpr int elem_bytes(int var) { return var == kVarFp8 || var == kVarInt8 ? 1 : 2; }

template <int HD, int EB>
struct Tile {
    static constexpr int kBytes = kBlock * HD * EB;  // one 16-token K or V tile
};

// The first `valid` tokens of a block.
struct FirstTokens {
    int valid;
    __device__ __forceinline__ bool operator()(int t) const { return t < valid; }
};

// The tokens whose bit is set.
struct TokenMask {
    uint32_t bits;
    __device__ __forceinline__ bool operator()(int t) const { return (bits >> t) & 1u; }
};

// Scored step: this lane's four logits (heads 2(lane & 3) and the next one of
// tokens lane / 4 and lane / 4 + 8) into the block's [16][gp] rows.
__device__ __forceinline__ void store_logits(float* lg, int gp, int lane, float s0, float s1, float s2, float s3) {
    const int h0 = (lane & 3) * 2;
    if (h0 < gp) {
        float* at = lg + (lane >> 2) * gp + h0;
        *reinterpret_cast<float2*>(at) = make_float2(s0, s1);
        *reinterpret_cast<float2*>(at + 8 * gp) = make_float2(s2, s3);
    }
}

__device__ __forceinline__ uint2 pack_bf16x4(float4 v) {
    return make_uint2((uint32_t)f32_to_bf16(v.x) | ((uint32_t)f32_to_bf16(v.y) << 16),
                      (uint32_t)f32_to_bf16(v.z) | ((uint32_t)f32_to_bf16(v.w) << 16));
}

// Tensor-core tile: S^T[16 tokens x 8 heads] = K[16 x HD] . Q^T[HD x 8] with
// mma.sync m16n8k16 (heads beyond G are zero columns), online softmax on the
// fragments, then O^T[HD x 8] += V^T[HD x 16] . P^T[16 x 8] (V^T by
// ldmatrix.trans, P^T by movmatrix.trans of the score fragments).
// With SCORED, a block's base-2 logits also go to `lg` ([16 tokens][gp] in
// global memory) and the sums take the weights before their rounding to bf16:
// the row's log-sum-exp then carries fp32 precision, which the weights
// recomputed from it need and the output (whose values are rounded to 8 bits
// anyway) does not mind.
template <int HD, bool SCORED = false>
struct MmaState {
    static constexpr int kK = HD / 16;
    uint32_t qb[kK][2];
    float o[kK][4];
    float m[2], l[2];

    template <class Params>
    __device__ __forceinline__ void begin_unit(const Params& p, int b, int h, int lane) {
        const int n = lane >> 2;
        const bool ok = n < p.G;
        const uint16_t* qrow = p.q + ((long long)b * p.Hq + (long long)h * p.G + (ok ? n : 0)) * HD;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
            const int dcol = kk * 16 + (lane & 3) * 2;
            qb[kk][0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow + dcol)) : 0u;
            qb[kk][1] = ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow + dcol + 8)) : 0u;
        }
#pragma unroll
        for (int mt = 0; mt < kK; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = kNegInf;
        l[0] = l[1] = 0.f;
    }

    // The fused decode step: q of the unit's heads from rotated rows [G][HD]
    // bf16 in shared memory (the RoPE warp's ring slot).
    template <class Params>
    __device__ __forceinline__ void begin_unit_from(const uint16_t* qrows, const Params& p, int /*h*/,
                                                    int lane) {
        const int n = lane >> 2;
        const bool ok = n < p.G;
        const uint16_t* qrow = qrows + (ok ? n : 0) * HD;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
            const int dcol = kk * 16 + (lane & 3) * 2;
            qb[kk][0] = ok ? *reinterpret_cast<const uint32_t*>(qrow + dcol) : 0u;
            qb[kk][1] = ok ? *reinterpret_cast<const uint32_t*>(qrow + dcol + 8) : 0u;
        }
#pragma unroll
        for (int mt = 0; mt < kK; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = kNegInf;
        l[0] = l[1] = 0.f;
    }

    template <class Seen>
    __device__ __forceinline__ void block(uint32_t kt, uint32_t vt, Seen seen, float sl2, int lane,
                                          float* lg = nullptr, int gp = 0) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        {
            // two accumulation chains (even / odd k-slices) halve the
            // dependent MMA latency
            float c1[4] = {0.f, 0.f, 0.f, 0.f};
            const int tok = (lane & 7) + ((lane >> 3) & 1) * 8;
            const int csel = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < kK; ++kk) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(kt + swz<HD>(tok, kk * 2 + csel), a0, a1, a2, a3);
                mma_bf16_16816(kk & 1 ? c1 : c, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] += c1[i];
        }
        const int t0 = lane >> 2, t1 = t0 + 8;
        float s0 = seen(t0) ? c[0] * sl2 : kNegInf;  // head 2*(lane&3),   token t0
        float s1 = seen(t0) ? c[1] * sl2 : kNegInf;  // head 2*(lane&3)+1, token t0
        float s2 = seen(t1) ? c[2] * sl2 : kNegInf;  // head 2*(lane&3),   token t1
        float s3 = seen(t1) ? c[3] * sl2 : kNegInf;  // head 2*(lane&3)+1, token t1
        if constexpr (SCORED) store_logits(lg, gp, lane, s0, s1, s2, s3);
        float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
        const float r0 = mn0 == kNegInf ? 0.f : mn0, r1 = mn1 == kNegInf ? 0.f : mn1;
        const float al0 = ex2(m[0] - r0), al1 = ex2(m[1] - r1);
        m[0] = mn0;
        m[1] = mn1;
        const float e0 = ex2(s0 - r0), e1 = ex2(s1 - r1), e2 = ex2(s2 - r0), e3 = ex2(s3 - r1);
        const uint32_t x0 = pack_bf16x2(e0, e1);
        const uint32_t x1 = pack_bf16x2(e2, e3);
        if constexpr (SCORED) {
            l[0] = l[0] * al0 + (e0 + e2);
            l[1] = l[1] * al1 + (e1 + e3);
        } else {
            // the sums use the same bf16-rounded weights the PV product uses
            l[0] = l[0] * al0 + (bf16_lo(x0) + bf16_lo(x1));
            l[1] = l[1] * al1 + (bf16_hi(x0) + bf16_hi(x1));
        }
        // the running max rarely moves once a few blocks are in: skip the
        // rescale when no lane's factor differs from 1
        if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < kK; ++mt) {
                o[mt][0] *= al0;
                o[mt][1] *= al1;
                o[mt][2] *= al0;
                o[mt][3] *= al1;
            }
        }
        const uint32_t b0 = movmatrix_trans(x0), b1 = movmatrix_trans(x1);
        {
            const int qd = lane >> 3;
            const int tok = (lane & 7) + (qd >> 1) * 8;
            const int csel = qd & 1;
#pragma unroll
            for (int mt = 0; mt < kK; ++mt) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4_trans(vt + swz<HD>(tok, mt * 2 + csel), a0, a1, a2, a3);
                mma_bf16_16816(o[mt], a0, a1, a2, a3, b0, b1);
            }
        }
    }

    // The warp's sums in every lane; then each() hands out this lane's outputs, not
    // yet divided by the sums: f(0 or 1 (head 2 (lane & 3) or the next), first
    // dim, kRun consecutive values).
    static constexpr int kRun = 1;
    __device__ __forceinline__ void sums() {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], sh);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], sh);
        }
    }
    template <class F>
    __device__ __forceinline__ void each(int lane, F f) const {
        const int r = lane >> 2;
#pragma unroll
        for (int mt = 0; mt < kK; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v[1] = {o[mt][e]};
                f(e & 1, mt * 16 + r + (e >> 1) * 8, v);
            }
    }

    // Reduce the per-thread sums and write (m, l, O) of this warp to smem.
    __device__ __forceinline__ void store(float* mbuf, float* lbuf, float* obuf, int G, int lane) {
        sums();
        const int h0 = (lane & 3) * 2, h1 = h0 + 1;
        if (lane < 4) {
            if (h0 < G) { mbuf[h0] = m[0]; lbuf[h0] = l[0]; }
            if (h1 < G) { mbuf[h1] = m[1]; lbuf[h1] = l[1]; }
        }
        const int r = lane >> 2;
#pragma unroll
        for (int mt = 0; mt < kK; ++mt) {
            if (h0 < G) {
                obuf[h0 * HD + mt * 16 + r] = o[mt][0];
                obuf[h0 * HD + mt * 16 + r + 8] = o[mt][2];
            }
            if (h1 < G) {
                obuf[h1 * HD + mt * 16 + r] = o[mt][1];
                obuf[h1 * HD + mt * 16 + r + 8] = o[mt][3];
            }
        }
    }
};

// Tensor-core tile over e4m3 (FP8) K/V tiles, the MMA tile's arithmetic in
// f16 (every e4m3 value is an f16 value, and f16 keeps 11 bits of the
// probabilities). S^T = K . Q^T: ldmatrix hands each lane four consecutive K
// bytes of a token row, which convert to two f16 pairs; within every 16-dim
// k-slice the lane's k slots (2c, 2c+1) and (2c+8, 2c+9) are taken to be dims
// (4c, 4c+1) and (4c+2, 4c+3), and Q's fragments are loaded in the same order,
// so the dot products are unchanged. O^T = V^T . P^T: each lane reads four
// bytes (dims 4j..4j+3) of token rows 2c, 2c+1, 2c+8, 2c+9, byte-permutes
// them into (token pair, dim) pairs and converts; the 16 O^T rows of a tile
// pair are dims 4(8t + r) + {0, 1} (even tile) and + {2, 3} (odd tile).
// K's per-head scale folds into the exponent scale, V's into the output.
template <int HD, bool SCORED = false>
struct Fp8State {
    static constexpr int kK = HD / 16;
    uint32_t qb[kK][2];
    float o[kK][4];
    float m[2], l[2];
    float sl2, vsc;

    template <class Params>
    __device__ __forceinline__ void begin_unit(const Params& p, int b, int h, int lane) {
        const int n = lane >> 2, c = lane & 3;
        const bool ok = n < p.G;
        const uint16_t* qrow = p.q + ((long long)b * p.Hq + (long long)h * p.G + (ok ? n : 0)) * HD;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
            const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(qrow + kk * 16 + 4 * c)) : make_uint2(0, 0);
            qb[kk][0] = pack_f16x2(bf16_lo(w.x), bf16_hi(w.x));  // dims 4c, 4c+1
            qb[kk][1] = pack_f16x2(bf16_lo(w.y), bf16_hi(w.y));  // dims 4c+2, 4c+3
        }
#pragma unroll
        for (int mt = 0; mt < kK; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = kNegInf;
        l[0] = l[1] = 0.f;
        sl2 = p.sl2 * __ldg(p.k_scale + h);
        vsc = __ldg(p.v_scale + h);
    }

    // The fused decode step: q of the unit's heads from rotated rows [G][HD]
    // bf16 in shared memory (the RoPE warp's ring slot), in the same order.
    template <class Params>
    __device__ __forceinline__ void begin_unit_from(const uint16_t* qrows, const Params& p, int h, int lane) {
        const int n = lane >> 2, c = lane & 3;
        const bool ok = n < p.G;
        const uint16_t* qrow = qrows + (ok ? n : 0) * HD;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
            const uint2 w = ok ? *reinterpret_cast<const uint2*>(qrow + kk * 16 + 4 * c) : make_uint2(0, 0);
            qb[kk][0] = pack_f16x2(bf16_lo(w.x), bf16_hi(w.x));
            qb[kk][1] = pack_f16x2(bf16_lo(w.y), bf16_hi(w.y));
        }
#pragma unroll
        for (int mt = 0; mt < kK; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = kNegInf;
        l[0] = l[1] = 0.f;
        sl2 = p.sl2 * __ldg(p.k_scale + h);
        vsc = __ldg(p.v_scale + h);
    }

    template <class Seen>
    __device__ __forceinline__ void block(uint32_t kt, uint32_t vt, Seen seen, float /*sl2 of bf16*/, int lane,
                                          float* lg = nullptr, int gp = 0) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        {
            float c1[4] = {0.f, 0.f, 0.f, 0.f};  // second accumulation chain (odd k-slices)
            const int mi = lane >> 3;
            const int tok = (lane & 7) + (mi & 1) * 8;
#pragma unroll
            for (int kp = 0; kp < kK / 2; ++kp) {
                uint32_t r0, r1, r2, r3;  // tokens g / g+8 of k-slices 2kp / 2kp+1
                ldsm_x4(kt + swz8<HD>(tok, 2 * kp + (mi >> 1)), r0, r1, r2, r3);
                mma_f16_16816(c, e4m3x2_to_f16x2(r0), e4m3x2_to_f16x2(r1), e4m3x2_to_f16x2(r0 >> 16),
                              e4m3x2_to_f16x2(r1 >> 16), qb[2 * kp][0], qb[2 * kp][1]);
                mma_f16_16816(c1, e4m3x2_to_f16x2(r2), e4m3x2_to_f16x2(r3), e4m3x2_to_f16x2(r2 >> 16),
                              e4m3x2_to_f16x2(r3 >> 16), qb[2 * kp + 1][0], qb[2 * kp + 1][1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] += c1[i];
        }
        const int t0 = lane >> 2, t1 = t0 + 8;
        float s0 = seen(t0) ? c[0] * sl2 : kNegInf;
        float s1 = seen(t0) ? c[1] * sl2 : kNegInf;
        float s2 = seen(t1) ? c[2] * sl2 : kNegInf;
        float s3 = seen(t1) ? c[3] * sl2 : kNegInf;
        if constexpr (SCORED) store_logits(lg, gp, lane, s0, s1, s2, s3);
        float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
        const float r0 = mn0 == kNegInf ? 0.f : mn0, r1 = mn1 == kNegInf ? 0.f : mn1;
        const float al0 = ex2(m[0] - r0), al1 = ex2(m[1] - r1);
        m[0] = mn0;
        m[1] = mn1;
        const float e0 = ex2(s0 - r0), e1 = ex2(s1 - r1), e2 = ex2(s2 - r0), e3 = ex2(s3 - r1);
        const uint32_t x0 = pack_f16x2(e0, e1);
        const uint32_t x1 = pack_f16x2(e2, e3);
        if constexpr (SCORED) {
            l[0] = l[0] * al0 + (e0 + e2);
            l[1] = l[1] * al1 + (e1 + e3);
        } else {
            l[0] = l[0] * al0 + (f16_lo(x0) + f16_lo(x1));
            l[1] = l[1] * al1 + (f16_hi(x0) + f16_hi(x1));
        }
        if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < kK; ++mt) {
                o[mt][0] *= al0;
                o[mt][1] *= al1;
                o[mt][2] *= al0;
                o[mt][3] *= al1;
            }
        }
        const uint32_t b0 = movmatrix_trans(x0), b1 = movmatrix_trans(x1);
        {
            const int g = lane >> 2, cc = lane & 3;
#pragma unroll
            for (int t = 0; t < kK / 2; ++t) {
                // dims 4j .. 4j+3, j = 8t + g, of token rows 2cc, 2cc+1, 2cc+8, 2cc+9
                const int chunk = 2 * t + (g >> 2), inb = (g & 3) * 4;
                const uint32_t w0 = lds32(vt + swz8<HD>(2 * cc, chunk) + inb);
                const uint32_t w1 = lds32(vt + swz8<HD>(2 * cc + 1, chunk) + inb);
                const uint32_t w2 = lds32(vt + swz8<HD>(2 * cc + 8, chunk) + inb);
                const uint32_t w3 = lds32(vt + swz8<HD>(2 * cc + 9, chunk) + inb);
                const uint32_t lo01 = __byte_perm(w0, w1, 0x5140), hi01 = __byte_perm(w0, w1, 0x7362);
                const uint32_t lo89 = __byte_perm(w2, w3, 0x5140), hi89 = __byte_perm(w2, w3, 0x7362);
                mma_f16_16816(o[2 * t], e4m3x2_to_f16x2(lo01), e4m3x2_to_f16x2(lo01 >> 16), e4m3x2_to_f16x2(lo89),
                              e4m3x2_to_f16x2(lo89 >> 16), b0, b1);
                mma_f16_16816(o[2 * t + 1], e4m3x2_to_f16x2(hi01), e4m3x2_to_f16x2(hi01 >> 16),
                              e4m3x2_to_f16x2(hi89), e4m3x2_to_f16x2(hi89 >> 16), b0, b1);
            }
        }
    }

    // Two blocks at once, the second's tiles `next` bytes behind the first's; seen(t):
    // token t of the 32. One maximum and one rescaling for both, and twice as many
    // products that do not depend on one another.
    template <class Seen>
    __device__ __forceinline__ void pair(uint32_t kt, uint32_t vt, uint32_t next, Seen seen, int lane) {
        float s[2][4];
        {
            const int mi = lane >> 3;
            const int tok = (lane & 7) + (mi & 1) * 8;
            float c[2][4] = {}, c1[2][4] = {};
#pragma unroll
            for (int kp = 0; kp < kK / 2; ++kp) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t r0, r1, r2, r3;
                    ldsm_x4(kt + x * next + swz8<HD>(tok, 2 * kp + (mi >> 1)), r0, r1, r2, r3);
                    mma_f16_16816(c[x], e4m3x2_to_f16x2(r0), e4m3x2_to_f16x2(r1), e4m3x2_to_f16x2(r0 >> 16),
                                  e4m3x2_to_f16x2(r1 >> 16), qb[2 * kp][0], qb[2 * kp][1]);
                    mma_f16_16816(c1[x], e4m3x2_to_f16x2(r2), e4m3x2_to_f16x2(r3), e4m3x2_to_f16x2(r2 >> 16),
                                  e4m3x2_to_f16x2(r3 >> 16), qb[2 * kp + 1][0], qb[2 * kp + 1][1]);
                }
            }
            const int t0 = lane >> 2;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[x][i] = seen(16 * x + t0 + 8 * (i >> 1)) ? (c[x][i] + c1[x][i]) * sl2 : kNegInf;
        }
        float mx0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
        float mx1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
        const float r0 = mn0 == kNegInf ? 0.f : mn0, r1 = mn1 == kNegInf ? 0.f : mn1;
        const float al0 = ex2(m[0] - r0), al1 = ex2(m[1] - r1);
        m[0] = mn0;
        m[1] = mn1;
        uint32_t b[2][2];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t x0 = pack_f16x2(ex2(s[x][0] - r0), ex2(s[x][1] - r1));
            const uint32_t x1 = pack_f16x2(ex2(s[x][2] - r0), ex2(s[x][3] - r1));
            l0 += f16_lo(x0) + f16_lo(x1);
            l1 += f16_hi(x0) + f16_hi(x1);
            b[x][0] = movmatrix_trans(x0);
            b[x][1] = movmatrix_trans(x1);
        }
        l[0] = l[0] * al0 + l0;
        l[1] = l[1] * al1 + l1;
        if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < kK; ++mt) {
                o[mt][0] *= al0;
                o[mt][1] *= al1;
                o[mt][2] *= al0;
                o[mt][3] *= al1;
            }
        }
        const int g = lane >> 2, cc = lane & 3;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t v = vt + x * next;
#pragma unroll
            for (int t = 0; t < kK / 2; ++t) {
                const int chunk = 2 * t + (g >> 2), inb = (g & 3) * 4;
                const uint32_t w0 = lds32(v + swz8<HD>(2 * cc, chunk) + inb);
                const uint32_t w1 = lds32(v + swz8<HD>(2 * cc + 1, chunk) + inb);
                const uint32_t w2 = lds32(v + swz8<HD>(2 * cc + 8, chunk) + inb);
                const uint32_t w3 = lds32(v + swz8<HD>(2 * cc + 9, chunk) + inb);
                const uint32_t lo01 = __byte_perm(w0, w1, 0x5140), hi01 = __byte_perm(w0, w1, 0x7362);
                const uint32_t lo89 = __byte_perm(w2, w3, 0x5140), hi89 = __byte_perm(w2, w3, 0x7362);
                mma_f16_16816(o[2 * t], e4m3x2_to_f16x2(lo01), e4m3x2_to_f16x2(lo01 >> 16), e4m3x2_to_f16x2(lo89),
                              e4m3x2_to_f16x2(lo89 >> 16), b[x][0], b[x][1]);
                mma_f16_16816(o[2 * t + 1], e4m3x2_to_f16x2(hi01), e4m3x2_to_f16x2(hi01 >> 16),
                              e4m3x2_to_f16x2(hi89), e4m3x2_to_f16x2(hi89 >> 16), b[x][0], b[x][1]);
            }
        }
    }

    // The warp's sums in every lane; then each() hands out this lane's outputs, not
    // yet divided by the sums: f(0 or 1 (head 2 (lane & 3) or the next), first
    // dim, kRun consecutive values).
    static constexpr int kRun = 4;
    __device__ __forceinline__ void sums() {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], sh);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], sh);
        }
    }
    template <class F>
    __device__ __forceinline__ void each(int lane, F f) const {
        const int r = lane >> 2;
#pragma unroll
        for (int t = 0; t < kK / 2; ++t)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float v[4] = {o[2 * t][w] * vsc, o[2 * t][2 + w] * vsc, o[2 * t + 1][w] * vsc, o[2 * t + 1][2 + w] * vsc};
                f(w, 4 * (8 * t + r), v);
            }
    }

    // Reduce the per-thread sums and write (m, l, O * v_scale) of this warp to smem.
    __device__ __forceinline__ void store(float* mbuf, float* lbuf, float* obuf, int G, int lane) {
        sums();
        const int h0 = (lane & 3) * 2, h1 = h0 + 1;
        if (lane < 4) {
            if (h0 < G) { mbuf[h0] = m[0]; lbuf[h0] = l[0]; }
            if (h1 < G) { mbuf[h1] = m[1]; lbuf[h1] = l[1]; }
        }
        const int r = lane >> 2;
#pragma unroll
        for (int t = 0; t < kK / 2; ++t) {
            const int d0 = 4 * (8 * t + r);
            if (h0 < G) {
                obuf[h0 * HD + d0] = o[2 * t][0] * vsc;
                obuf[h0 * HD + d0 + 1] = o[2 * t][2] * vsc;
                obuf[h0 * HD + d0 + 2] = o[2 * t + 1][0] * vsc;
                obuf[h0 * HD + d0 + 3] = o[2 * t + 1][2] * vsc;
            }
            if (h1 < G) {
                obuf[h1 * HD + d0] = o[2 * t][1] * vsc;
                obuf[h1 * HD + d0 + 1] = o[2 * t][3] * vsc;
                obuf[h1 * HD + d0 + 2] = o[2 * t + 1][1] * vsc;
                obuf[h1 * HD + d0 + 3] = o[2 * t + 1][3] * vsc;
            }
        }
    }
};

// Tensor-core tile over INT8 K/V tiles quantised in 64-token groups: the e4m3
// tile's data movement and fragment orders. K's codes enter the MMAs as the f16
// values 1152 + code (a byte permute, exact); the bias comes back off the scores,
// 1152 times the sum of the head's q (a constant per head, folded into the scaling
// FMA). V's codes enter as themselves, one subtraction a pair: O adds up over
// hundreds of blocks, and the tensor cores cut each sum towards zero, so that with
// the bias in it O lost a part of 1152 times the probabilities in every block (a
// hundredth of the outputs behind a window of 8,192; 66 thousandths where the
// weights are equal). A block's
// codes stand for code * a / 127, a the maximum of its group (one per block
// and head, staged with the tile): K's factor multiplies the block's scores;
// V's factor is taken relative to a reference factor of the warp (the first
// block's, raised, with a rescale of O, when a block's factor exceeds it
// 256-fold) and multiplies the f16 probabilities of the block (at most 256,
// so within f16's range), while the running sum keeps the unscaled ones. O
// times the reference is the output.
template <int HD>
struct Int8State {
    static constexpr int kK = HD / 16;
    static constexpr uint32_t kFlip = 0x80808080u;  // sign bits: codes to offset binary
    static constexpr uint32_t kLo = 0x4140u, kHi = 0x4342u;
    static constexpr float kBias = 1152.f;
    uint32_t qb[kK][2];
    float o[kK][4];
    float m[2], l[2];
    float koff[2];  // kBias * sum of q over the dims, for this lane's two heads
    float sl2, vref, rvref;

    template <class Params>
    __device__ __forceinline__ void reset(const Params& p, int lane) {
#pragma unroll
        for (int mt = 0; mt < kK; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m[0] = m[1] = kNegInf;
        l[0] = l[1] = 0.f;
        sl2 = p.sl2 * (1.f / 127.f);
        vref = 0.f;
        rvref = 0.f;
        // q's sum per head: lane (n, c) holds dims 4c..4c+3 of every 16-dim
        // slice of head n; the quad reduces, then each lane takes the sums of
        // the heads its score columns hold (2c and 2c + 1)
        float qs = 0.f;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk)
            qs += (f16_lo(qb[kk][0]) + f16_hi(qb[kk][0])) + (f16_lo(qb[kk][1]) + f16_hi(qb[kk][1]));
        qs += __shfl_xor_sync(0xffffffffu, qs, 1);
        qs += __shfl_xor_sync(0xffffffffu, qs, 2);
        koff[0] = kBias * __shfl_sync(0xffffffffu, qs, 8 * (lane & 3));
        koff[1] = kBias * __shfl_sync(0xffffffffu, qs, 8 * (lane & 3) + 4);
    }

    template <class Params>
    __device__ __forceinline__ void begin_unit(const Params& p, int b, int h, int lane) {
        const int n = lane >> 2, c = lane & 3;
        const bool ok = n < p.G;
        const uint16_t* qrow = p.q + ((long long)b * p.Hq + (long long)h * p.G + (ok ? n : 0)) * HD;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
            const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(qrow + kk * 16 + 4 * c)) : make_uint2(0, 0);
            qb[kk][0] = pack_f16x2(bf16_lo(w.x), bf16_hi(w.x));  // dims 4c, 4c+1
            qb[kk][1] = pack_f16x2(bf16_lo(w.y), bf16_hi(w.y));  // dims 4c+2, 4c+3
        }
        reset(p, lane);
    }

    template <class Params>
    __device__ __forceinline__ void begin_unit_from(const uint16_t*, const Params& p, int, int lane) {
        reset(p, lane);
    }

    template <class Seen>
    __device__ __forceinline__ void block(uint32_t kt, uint32_t vt, Seen seen, int lane, float ak, float av) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        {
            float c1[4] = {0.f, 0.f, 0.f, 0.f};  // second accumulation chain (odd k-slices)
            const int mi = lane >> 3;
            const int tok = (lane & 7) + (mi & 1) * 8;
#pragma unroll
            for (int kp = 0; kp < kK / 2; ++kp) {
                uint32_t r0, r1, r2, r3;  // tokens g / g+8 of k-slices 2kp / 2kp+1
                ldsm_x4(kt + swz8<HD>(tok, 2 * kp + (mi >> 1)), r0, r1, r2, r3);
                r0 ^= kFlip;
                r1 ^= kFlip;
                r2 ^= kFlip;
                r3 ^= kFlip;
                mma_f16_16816(c, i8x2_to_f16x2_biased(r0, kLo), i8x2_to_f16x2_biased(r1, kLo),
                              i8x2_to_f16x2_biased(r0, kHi), i8x2_to_f16x2_biased(r1, kHi), qb[2 * kp][0],
                              qb[2 * kp][1]);
                mma_f16_16816(c1, i8x2_to_f16x2_biased(r2, kLo), i8x2_to_f16x2_biased(r3, kLo),
                              i8x2_to_f16x2_biased(r2, kHi), i8x2_to_f16x2_biased(r3, kHi), qb[2 * kp + 1][0],
                              qb[2 * kp + 1][1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] += c1[i];
        }
        const float ks = sl2 * ak;  // scale * log2(e) * a_k / 127
        const float kb0 = ks * koff[0], kb1 = ks * koff[1];
        const int t0 = lane >> 2, t1 = t0 + 8;
        float s0 = seen(t0) ? fmaf(c[0], ks, -kb0) : kNegInf;
        float s1 = seen(t0) ? fmaf(c[1], ks, -kb1) : kNegInf;
        float s2 = seen(t1) ? fmaf(c[2], ks, -kb0) : kNegInf;
        float s3 = seen(t1) ? fmaf(c[3], ks, -kb1) : kNegInf;
        float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
        const float r0 = mn0 == kNegInf ? 0.f : mn0, r1 = mn1 == kNegInf ? 0.f : mn1;
        float al0 = ex2(m[0] - r0), al1 = ex2(m[1] - r1);
        m[0] = mn0;
        m[1] = mn1;
        const float p0 = ex2(s0 - r0), p1 = ex2(s1 - r1), p2 = ex2(s2 - r0), p3 = ex2(s3 - r1);
        l[0] = l[0] * al0 + (p0 + p2);
        l[1] = l[1] * al1 + (p1 + p3);
        // V's factor relative to the reference (the same for every lane)
        const float fv = av * (1.f / 127.f);
        float ov0 = al0, ov1 = al1;  // O's factors for this block
        if (fv > vref * 256.f) {
            const float f = vref * (1.f / fv);  // 0 for the first nonzero factor (O is still 0)
            ov0 *= f;
            ov1 *= f;
            vref = fv;
            rvref = 1.f / fv;
        }
        const float rel = fv * rvref;
        const uint32_t x0 = pack_f16x2(p0 * rel, p1 * rel);
        const uint32_t x1 = pack_f16x2(p2 * rel, p3 * rel);
        if (__any_sync(0xffffffffu, ov0 != 1.f || ov1 != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < kK; ++mt) {
                o[mt][0] *= ov0;
                o[mt][1] *= ov1;
                o[mt][2] *= ov0;
                o[mt][3] *= ov1;
            }
        }
        const uint32_t b0 = movmatrix_trans(x0), b1 = movmatrix_trans(x1);
        {
            const int g = lane >> 2, cc = lane & 3;
#pragma unroll
            for (int t = 0; t < kK / 2; ++t) {
                // dims 4j .. 4j+3, j = 8t + g, of token rows 2cc, 2cc+1, 2cc+8, 2cc+9
                const int chunk = 2 * t + (g >> 2), inb = (g & 3) * 4;
                const uint32_t w0 = lds32(vt + swz8<HD>(2 * cc, chunk) + inb);
                const uint32_t w1 = lds32(vt + swz8<HD>(2 * cc + 1, chunk) + inb);
                const uint32_t w2 = lds32(vt + swz8<HD>(2 * cc + 8, chunk) + inb);
                const uint32_t w3 = lds32(vt + swz8<HD>(2 * cc + 9, chunk) + inb);
                const uint32_t lo01 = __byte_perm(w0, w1, 0x5140) ^ kFlip, hi01 = __byte_perm(w0, w1, 0x7362) ^ kFlip;
                const uint32_t lo89 = __byte_perm(w2, w3, 0x5140) ^ kFlip, hi89 = __byte_perm(w2, w3, 0x7362) ^ kFlip;
                mma_f16_16816(o[2 * t], i8x2_to_f16x2(lo01, kLo), i8x2_to_f16x2(lo01, kHi),
                              i8x2_to_f16x2(lo89, kLo), i8x2_to_f16x2(lo89, kHi), b0, b1);
                mma_f16_16816(o[2 * t + 1], i8x2_to_f16x2(hi01, kLo), i8x2_to_f16x2(hi01, kHi),
                              i8x2_to_f16x2(hi89, kLo), i8x2_to_f16x2(hi89, kHi), b0, b1);
            }
        }
    }

    // Two blocks at once, as Fp8State::pair; each with its own factors (av 0 where a
    // block is absent: none of its tokens is seen).
    template <class Seen>
    __device__ __forceinline__ void pair(uint32_t kt, uint32_t vt, uint32_t next, Seen seen, int lane, float ak0, float ak1,
                                         float av0, float av1) {
        float s[2][4];
        {
            const int mi = lane >> 3;
            const int tok = (lane & 7) + (mi & 1) * 8;
            float c[2][4] = {}, c1[2][4] = {};
#pragma unroll
            for (int kp = 0; kp < kK / 2; ++kp) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t r0, r1, r2, r3;
                    ldsm_x4(kt + x * next + swz8<HD>(tok, 2 * kp + (mi >> 1)), r0, r1, r2, r3);
                    r0 ^= kFlip;
                    r1 ^= kFlip;
                    r2 ^= kFlip;
                    r3 ^= kFlip;
                    mma_f16_16816(c[x], i8x2_to_f16x2_biased(r0, kLo), i8x2_to_f16x2_biased(r1, kLo),
                                  i8x2_to_f16x2_biased(r0, kHi), i8x2_to_f16x2_biased(r1, kHi), qb[2 * kp][0],
                                  qb[2 * kp][1]);
                    mma_f16_16816(c1[x], i8x2_to_f16x2_biased(r2, kLo), i8x2_to_f16x2_biased(r3, kLo),
                                  i8x2_to_f16x2_biased(r2, kHi), i8x2_to_f16x2_biased(r3, kHi), qb[2 * kp + 1][0],
                                  qb[2 * kp + 1][1]);
                }
            }
            const int t0 = lane >> 2;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float ks = sl2 * (x ? ak1 : ak0);  // scale * log2(e) * a_k / 127
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[x][i] = seen(16 * x + t0 + 8 * (i >> 1)) ? fmaf(c[x][i] + c1[x][i], ks, -(ks * koff[i & 1])) : kNegInf;
            }
        }
        float mx0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
        float mx1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        }
        const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
        const float r0 = mn0 == kNegInf ? 0.f : mn0, r1 = mn1 == kNegInf ? 0.f : mn1;
        const float al0 = ex2(m[0] - r0), al1 = ex2(m[1] - r1);
        m[0] = mn0;
        m[1] = mn1;
        // the larger of the blocks' V factors moves the reference (the same for every lane)
        const float fv = fmaxf(av0, av1) * (1.f / 127.f);
        float ov0 = al0, ov1 = al1;  // O's factors for these blocks
        if (fv > vref * 256.f) {
            const float f = vref * (1.f / fv);  // 0 for the first nonzero factor (O is still 0)
            ov0 *= f;
            ov1 *= f;
            vref = fv;
            rvref = 1.f / fv;
        }
        uint32_t b[2][2];
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float p0 = ex2(s[x][0] - r0), p1 = ex2(s[x][1] - r1), p2 = ex2(s[x][2] - r0), p3 = ex2(s[x][3] - r1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            const float rel = (x ? av1 : av0) * (1.f / 127.f) * rvref;
            const uint32_t x0 = pack_f16x2(p0 * rel, p1 * rel), x1 = pack_f16x2(p2 * rel, p3 * rel);
            b[x][0] = movmatrix_trans(x0);
            b[x][1] = movmatrix_trans(x1);
        }
        l[0] = l[0] * al0 + l0;
        l[1] = l[1] * al1 + l1;
        if (__any_sync(0xffffffffu, ov0 != 1.f || ov1 != 1.f)) {
#pragma unroll
            for (int mt = 0; mt < kK; ++mt) {
                o[mt][0] *= ov0;
                o[mt][1] *= ov1;
                o[mt][2] *= ov0;
                o[mt][3] *= ov1;
            }
        }
        const int g = lane >> 2, cc = lane & 3;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t v = vt + x * next;
#pragma unroll
            for (int t = 0; t < kK / 2; ++t) {
                const int chunk = 2 * t + (g >> 2), inb = (g & 3) * 4;
                const uint32_t w0 = lds32(v + swz8<HD>(2 * cc, chunk) + inb);
                const uint32_t w1 = lds32(v + swz8<HD>(2 * cc + 1, chunk) + inb);
                const uint32_t w2 = lds32(v + swz8<HD>(2 * cc + 8, chunk) + inb);
                const uint32_t w3 = lds32(v + swz8<HD>(2 * cc + 9, chunk) + inb);
                const uint32_t lo01 = __byte_perm(w0, w1, 0x5140) ^ kFlip, hi01 = __byte_perm(w0, w1, 0x7362) ^ kFlip;
                const uint32_t lo89 = __byte_perm(w2, w3, 0x5140) ^ kFlip, hi89 = __byte_perm(w2, w3, 0x7362) ^ kFlip;
                mma_f16_16816(o[2 * t], i8x2_to_f16x2(lo01, kLo), i8x2_to_f16x2(lo01, kHi),
                              i8x2_to_f16x2(lo89, kLo), i8x2_to_f16x2(lo89, kHi), b[x][0], b[x][1]);
                mma_f16_16816(o[2 * t + 1], i8x2_to_f16x2(hi01, kLo), i8x2_to_f16x2(hi01, kHi),
                              i8x2_to_f16x2(hi89, kLo), i8x2_to_f16x2(hi89, kHi), b[x][0], b[x][1]);
            }
        }
    }

    // The warp's sums in every lane; then each() hands out this lane's outputs, not
    // yet divided by the sums: f(0 or 1 (head 2 (lane & 3) or the next), first
    // dim, kRun consecutive values).
    static constexpr int kRun = 4;
    __device__ __forceinline__ void sums() {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], sh);
            l[1] += __shfl_xor_sync(0xffffffffu, l[1], sh);
        }
    }
    template <class F>
    __device__ __forceinline__ void each(int lane, F f) const {
        const int r = lane >> 2;
#pragma unroll
        for (int t = 0; t < kK / 2; ++t)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float v[4] = {o[2 * t][w] * vref, o[2 * t][2 + w] * vref, o[2 * t + 1][w] * vref, o[2 * t + 1][2 + w] * vref};
                f(w, 4 * (8 * t + r), v);
            }
    }

    // Reduce the per-thread sums and write (m, l, O * reference) of this warp to smem.
    __device__ __forceinline__ void store(float* mbuf, float* lbuf, float* obuf, int G, int lane) {
        sums();
        const int h0 = (lane & 3) * 2, h1 = h0 + 1;
        if (lane < 4) {
            if (h0 < G) { mbuf[h0] = m[0]; lbuf[h0] = l[0]; }
            if (h1 < G) { mbuf[h1] = m[1]; lbuf[h1] = l[1]; }
        }
        const int r = lane >> 2;
#pragma unroll
        for (int t = 0; t < kK / 2; ++t) {
            const int d0 = 4 * (8 * t + r);
            if (h0 < G) {
                obuf[h0 * HD + d0] = o[2 * t][0] * vref;
                obuf[h0 * HD + d0 + 1] = o[2 * t][2] * vref;
                obuf[h0 * HD + d0 + 2] = o[2 * t + 1][0] * vref;
                obuf[h0 * HD + d0 + 3] = o[2 * t + 1][2] * vref;
            }
            if (h1 < G) {
                obuf[h1 * HD + d0] = o[2 * t][1] * vref;
                obuf[h1 * HD + d0 + 1] = o[2 * t][3] * vref;
                obuf[h1 * HD + d0 + 2] = o[2 * t + 1][1] * vref;
                obuf[h1 * HD + d0 + 3] = o[2 * t + 1][3] * vref;
            }
        }
    }
};

}  // namespace mi
