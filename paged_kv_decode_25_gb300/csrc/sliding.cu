// mi_paged_decode_attention_sliding: decode attention in which a token sees its
// sequence's first `sinks` tokens and its newest `window` ones. With n tokens held,
//   out = sum_t softmax_t(scale <q, K_t>) V_t,  t < n and (t < sinks or t >= n - window);
// blocks without such a token are neither copied nor looked up, so they may have
// been given back.
//
// Bound by the bytes in sight, which the window limits: a (request, KV head) has a
// few dozen blocks, not thousands, and what a launch costs around its streaming
// (the plan, the first copies, the ends of the work) weighs as much as the bytes.
// So a warp works by itself: it takes a piece, some consecutive blocks of a
// (request, head), looks the blocks up, copies them through a ring of its own (TMA,
// one mbarrier a stage), runs the decode tiles over them and writes the result,
// with no barrier among warps. A (request, head) of one piece is done then; of the
// others the warp that stores the last piece adds all of them up by their
// log-sum-exps, counted in a word per (request, head).
#include <atomic>
#include <chrono>
#include <cmath>
#include <random>

#include "batch.cuh"
#include "common.cuh"
#include "decode_tiles.cuh"
#include "sliding.cuh"
#include "tma.cuh"

namespace mi {
namespace {

constexpr int kSlideWarps = 4;

template <int HD, int VAR>
struct SlideShape {
    static constexpr int kTile = Tile<HD, elem_bytes(VAR)>::kBytes;
    static constexpr int kStages = 16384 / (2 * kTile) < 4 ? 16384 / (2 * kTile) : 4;
    static constexpr int kBlocksPerSm = 3;
    static constexpr int kSmem = kSlideWarps * kStages * 2 * kTile + 1024;  // slack to align the tiles
};

// Pieces that have partial results, at most, per warp of the grid.
constexpr int kSplitPerWarp = 8;
// A piece's own cost (its queries, its output, finding the next), in blocks, and
// that of adding up one piece at a (request, head)'s end.
constexpr float kPieceCost = 2.f, kMergeCost = 0.1f;

struct SlideParams {
    const uint16_t* q;             // [B][Hq][HD]
    const int32_t* block_tables;   // [B][mbps]
    const int32_t* context_lens;   // [B]
    uint16_t* out;                 // [B][Hq][HD]
    unsigned long long* words;     // [most]: at a split unit's first piece: epoch | pieces stored
    float* part;                   // [most][slot_floats] normalised output [G][HD], log2-sum-exps [G]
    unsigned long long epoch;      // distinct per call
    const float* k_scale;          // [Hkv] e4m3 caches
    const float* v_scale;
    const float* k_amax;           // [num_blocks][Hkv] INT8 caches
    const float* v_amax;
    int32_t* dev_err;
    int B, Hq, Hkv, G, num_blocks, mbps, window, sinks, most, slot_floats;
    float sl2;                     // scale * log2(e)
    float flow;                    // a block's time at full memory rate over its time in a warp, times all warps
    long long wait_ns;
    int withhold;                  // failure-detection test: each warp withholds its first copy
};

__device__ __forceinline__ Sight sight_of(const SlideParams& p, int b) {
    const int n = __ldg(p.context_lens + b), cap = p.mbps * kBlock;
    return Sight(n < 0 ? 0 : (n > cap ? cap : n), p.window, p.sinks);
}

// The blocks of a piece, chosen by every block of the launch alike: lane i tries
// i + 1 (and 32 + 15 i) pieces for the largest unit. Warps take whole pieces in
// turn; full rounds run at the memory's rate, in the last one a warp's own time may
// show, and so may the end of the unit with the most pieces.
__device__ int piece_blocks(const SlideParams& p, int warps, float blocks, float units, int largest, int lane) {
    const float all = blocks * p.flow;  // time of all blocks at the memory's rate, in a warp's block times
    float best = 3.0e38f, step = (float)largest;
    const float floor_step = fmaxf(1.f, ceilf(2.f * blocks / ((float)kSplitPerWarp * (float)warps)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float np = i == 0 ? (float)(lane + 1) : (float)(32 + 15 * lane);
        const float s = fmaxf(floor_step, ceilf((float)largest / np));
        const float most = ceilf((float)largest / s);
        // pieces: those of units of the largest size, and half a piece more than their share for the others
        const float even = units * (float)largest;
        const float pieces = even > 0.f ? units * most * (blocks / even) + 0.5f * units * (1.f - blocks / even) : 1.f;
        const float rounds = fmaxf(pieces, units) / (float)warps, full = floorf(rounds);
        const float cost = (full > 0.f ? full / rounds * all : 0.f) +
                           fmaxf(s + kPieceCost, (rounds - full) / rounds * all) + (most > 1.f ? kMergeCost * most : 0.f) +
                           0.01f * kPieceCost * rounds;
        if (cost < best) {
            best = cost;
            step = s;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xffffffffu, best, o), t = __shfl_xor_sync(0xffffffffu, step, o);
        if (c < best || (c == best && t < step)) {
            best = c;
            step = t;
        }
    }
    return (int)step;
}

// Whether this warp, its partial result written, is the last one of a unit of np
// pieces. The count is a word at the unit's first piece: high 48 bits the call's
// epoch, low 16 the pieces stored, so a word of another call counts as zero; the
// last piece hands it back as zero, so a captured call can be replayed.
__device__ __forceinline__ bool last_piece(const SlideParams& p, int slot, int np, int lane) {
    __syncwarp();
    int last = 0;
    if (lane == 0) {
        unsigned long long* wd = p.words + slot;
        const unsigned long long e48 = p.epoch & 0xFFFFFFFFFFFFull;
        unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(wd), nw, got;
        for (;;) {
            nw = ((old >> 16) == e48) ? old + 1 : ((e48 << 16) | 1ull);
            // this warp's partial result before the count, the others' after it
            asm volatile("atom.acq_rel.gpu.global.cas.b64 %0, [%1], %2, %3;"
                         : "=l"(got) : "l"(wd), "l"(old), "l"(nw) : "memory");
            if (got == old) break;
            old = got;
        }
        last = (int)(nw & 0xFFFFull) == np;
        if (last) *reinterpret_cast<volatile unsigned long long*>(wd) = 0ull;
    }
    last = __shfl_sync(0xffffffffu, last, 0);
    __syncwarp();
    return last != 0;
}

// The unit's output from its np pieces, in order: weights 2^(lse - M) over their
// sum, a lane per piece; then four outputs a lane and 512 bytes of a piece at a
// time, sixteen loads in flight.
template <int HD>
__device__ void merge_unit(const SlideParams& p, int b, int h, int slot, int np, int lane) {
    const float* part = p.part + (long long)slot * p.slot_floats;
    const int outs = p.G * HD;
    float top[kMaxG], den[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
        top[g] = kNegInf;
        if (g < p.G)
            for (int i = lane; i < np; i += 32) top[g] = fmaxf(top[g], __ldcg(part + (long long)i * p.slot_floats + outs + g));
    }
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top[g] = fmaxf(top[g], __shfl_xor_sync(0xffffffffu, top[g], o));
        den[g] = 0.f;
        if (top[g] == kNegInf) top[g] = 0.f;  // nothing in sight: weights 0
        if (g < p.G)
            for (int i = lane; i < np; i += 32) den[g] += exp2f(__ldcg(part + (long long)i * p.slot_floats + outs + g) - top[g]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den[g] += __shfl_xor_sync(0xffffffffu, den[g], o);
        den[g] = den[g] > 0.f ? 1.f / den[g] : 0.f;
    }
    uint16_t* out = p.out + ((long long)b * p.Hq + (long long)h * p.G) * HD;
    for (int k0 = 4 * lane; k0 < outs; k0 += 512) {  // up to four groups of 128 outputs
        float4 acc[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < np; ++i) {
            const float* at = part + (long long)i * p.slot_floats;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int x = k0 + 128 * k;
                if (x < outs) {
                    const int g = x / HD;
                    float t = top[0], d = den[0];
#pragma unroll
                    for (int e = 1; e < kMaxG; ++e)
                        if (g == e) {
                            t = top[e];
                            d = den[e];
                        }
                    const float w = exp2f(__ldcg(at + outs + g) - t) * d;
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(at + x));
                    acc[k].x += w * v.x;
                    acc[k].y += w * v.y;
                    acc[k].z += w * v.z;
                    acc[k].w += w * v.w;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k0 + 128 * k < outs) *reinterpret_cast<uint2*>(out + k0 + 128 * k) = pack_bf16x4(acc[k]);
    }
}

template <int HD, int VAR>
struct TileOf;
template <int HD>
struct TileOf<HD, kVarMma> { using T = MmaState<HD>; };
template <int HD>
struct TileOf<HD, kVarFp8> { using T = Fp8State<HD>; };
template <int HD>
struct TileOf<HD, kVarInt8> { using T = Int8State<HD>; };

template <int HD, int VAR>
__global__ void __launch_bounds__(kSlideWarps * 32, SlideShape<HD, VAR>::kBlocksPerSm)
    slide_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const SlideParams p) {
    using Shape = SlideShape<HD, VAR>;
    constexpr int S = Shape::kStages, kTile = Shape::kTile, kThreads = kSlideWarps * 32;
    constexpr bool kInt8 = VAR == kVarInt8, kFp8 = VAR == kVarFp8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long bars[kSlideWarps * S];
    __shared__ long long sums[flat_words(kThreads)], split_sums[flat_words(kThreads)];
    __shared__ long long red[2][kSlideWarps];
    __shared__ int red_top[kSlideWarps];
    __shared__ int held[kFlatOneWarp], first[kFlatOneWarp + 1], first_split[kFlatOneWarp];  // usual batches
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t full = smem_u32(bars) + warp * S * 8;
    const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + (uint32_t)(warp * S * 2 * kTile);
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(full + 8 * i, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    // ---------------------------------------------------------- the plan --
    const bool small = p.B <= kFlatOneWarp;
    long long blocks = 0, units = 0;  // (head, block)s in sight; (request, head)s with any
    int largest = 0;
    for (int b = tid; b < p.B; b += kThreads) {
        const int n = __ldg(p.context_lens + b);
        const int nb = sight_of(p, b).blocks;
        if (small) held[b] = nb;
        blocks += (long long)p.Hkv * nb;
        units += nb > 0 ? p.Hkv : 0;
        largest = max(largest, nb);
        if (b % (int)gridDim.x == (int)blockIdx.x) {
            if (n > p.mbps * kBlock) raise_err(p.dev_err, MI_DEVERR_BAD_CONTEXT);
            if (n <= 0) {  // no token: a zero row
                uint4* row = reinterpret_cast<uint4*>(p.out + (long long)b * p.Hq * HD);
                for (int i = 0; i < p.Hq * HD / 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
        units += __shfl_xor_sync(0xffffffffu, units, o);
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    }
    if (lane == 0) {
        red[0][warp] = blocks;
        red[1][warp] = units;
        red_top[warp] = largest;
    }
    __syncthreads();
    blocks = units = 0;
    for (int i = 0; i < kSlideWarps; ++i) {
        blocks += red[0][i];
        units += red[1][i];
        largest = max(largest, red_top[i]);
    }
    if (largest == 0) return;
    const int warps = gridDim.x * kSlideWarps;
    const int step = piece_blocks(p, warps, (float)blocks, (float)units, largest, lane);
    auto pieces_of = [&](int nb) { return (nb + step - 1) / step; };
    auto pieces = [&](int b) { return (long long)p.Hkv * pieces_of(sight_of(p, b).blocks); };
    auto splits = [&](int b) {
        const int np = pieces_of(sight_of(p, b).blocks);
        return np > 1 ? (long long)p.Hkv * np : 0LL;
    };
    long long total;
    if (small) {
        if (warp == 0) {
            const int per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
            int v = 0, w = 0;
            for (int b = b0; b < b1; ++b) {
                const int np = pieces_of(held[b]);
                v += p.Hkv * np;
                w += np > 1 ? p.Hkv * np : 0;
            }
            int x = v, y = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int s = __shfl_up_sync(0xffffffffu, x, o), t = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) {
                    x += s;
                    y += t;
                }
            }
            if (lane == 31) first[p.B] = x;
            x -= v;
            y -= w;
            for (int b = b0; b < b1; ++b) {
                const int np = pieces_of(held[b]);
                first[b] = x;
                first_split[b] = y;
                x += p.Hkv * np;
                y += np > 1 ? p.Hkv * np : 0;
            }
        }
        __syncthreads();
        total = first[p.B];
    } else {
        total = flat_scan(p.B, pieces, sums);
        (void)flat_scan(p.B, splits, split_sums);
    }
    // ---------------------------------------------------------- the pieces --
    struct Piece {
        long long x;
        int b, h, i, np, slot;  // piece i of the np of (request, head); the first one's partial result
        int j, j1;              // blocks in sight j .. j1 - 1
    };
    auto piece = [&](long long x) {
        Piece c;
        c.x = x;
        c.b = c.h = c.i = c.j = c.j1 = c.slot = 0;
        c.np = 1;
        if (x < total) {
            int o, nb;
            if (small) {
                int lo = 0, hi = p.B;  // first[lo] <= x < first[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (first[mid] <= (int)x) lo = mid;
                    else hi = mid;
                }
                c.b = lo;
                nb = held[lo];
                o = (int)x - first[lo];
                c.slot = first_split[lo];
            } else {
                long long before;
                c.b = flat_find(p.B, pieces, sums, x, before);
                nb = sight_of(p, c.b).blocks;
                o = (int)(x - before);
                c.slot = (int)flat_before(p.B, splits, split_sums, c.b);
            }
            c.np = pieces_of(nb);
            c.h = o / c.np;
            c.i = o - c.h * c.np;
            c.slot += c.h * c.np;
            // equal shares of the unit's blocks
            c.j = (int)((long long)nb * c.i / c.np);
            c.j1 = (int)((long long)nb * (c.i + 1) / c.np);
        }
        return c;
    };
    const uint64_t policy = l2_policy_evict_first();
    // the issuing side runs up to S blocks ahead, across pieces; table entries (and
    // an INT8 block's maxima) come 32 at a time
    Piece in = piece((long long)blockIdx.x * kSlideWarps + warp);
    Sight in_sight = sight_of(p, in.b);
    int entry = -1, base = 0;
    float ka = 0.f, va = 0.f;
    auto fetch = [&]() {
        base = in.j;
        entry = -1;
        ka = va = 0.f;
        if (in.x < total && in.j + lane < in.j1) {
            entry = __ldg(p.block_tables + (long long)in.b * p.mbps + in_sight.column(in.j + lane));
            if (kInt8 && entry >= 0 && entry < p.num_blocks) {
                ka = __ldg(p.k_amax + (long long)entry * p.Hkv + in.h);
                va = __ldg(p.v_amax + (long long)entry * p.Hkv + in.h);
            }
        }
    };
    fetch();
    uint32_t issued = 0, copied = 0, phase = 0;  // stages used; bit i: stage i holds a block; its parity
    float ks_of[kInt8 ? S : 1], vs_of[kInt8 ? S : 1];
    bool withhold = p.withhold != 0;
    auto issue = [&](uint32_t st) {
        if (in.x >= total) return;
        const int blk = __shfl_sync(0xffffffffu, entry, in.j - base);
        if constexpr (kInt8) {
            const float a = __shfl_sync(0xffffffffu, ka, in.j - base), v = __shfl_sync(0xffffffffu, va, in.j - base);
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (st == (uint32_t)i) {
                    ks_of[i] = a;
                    vs_of[i] = v;
                }
        }
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (lane == 0) {
            if (!ok) {
                raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
            } else if (!withhold) {
                const uint32_t bar = full + 8 * st, dst = ring + st * 2 * kTile;
                const int y = (blk * p.Hkv + in.h) * (kTile / 128);
                mbar_arrive_expect_tx(bar, 2 * kTile);
                tma_load_2d(dst, &tmk, bar, 0, y, policy);
                tma_load_2d(dst + kTile, &tmv, bar, 0, y, policy);
            }
        }
        withhold = false;
        copied = ok ? copied | (1u << st) : copied & ~(1u << st);
        ++issued;
        if (++in.j == in.j1) {
            in = piece(in.x + warps);
            in_sight = sight_of(p, in.b);
            fetch();
        } else if (in.j - base == 32) {
            fetch();
        }
    };
    __syncwarp();
    Piece c = in;
    for (int i = 0; i < S; ++i) issue((uint32_t)i);
    uint32_t taken = 0;
    bool dead = false;
    typename TileOf<HD, VAR>::T st;
    while (!dead && c.x < total) {
        const Sight sight = sight_of(p, c.b);
        st.begin_unit(p, c.b, c.h, lane);
        for (int j = c.j; j < c.j1; ++j, ++taken) {
            const uint32_t sg = taken % S;
            if ((copied >> sg) & 1u) {
                if (!wait_warp(full + 8 * sg, (phase >> sg) & 1u, p.wait_ns)) {
                    if (lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
                    dead = true;
                    break;
                }
                phase ^= 1u << sg;
                const uint32_t kt = ring + sg * 2 * kTile, vt = kt + kTile;
                const uint32_t seen = sight.mask(sight.column(j));
                if (!kInt8 && seen != 0xFFFFu) {
                    // rows out of sight may hold any bits: zero V there (INT8 codes are always finite)
                    constexpr int kChunks = HD * elem_bytes(VAR) / 16;
                    for (int i = lane; i < kBlock * kChunks; i += 32) {
                        const int row = i / kChunks, ch = i % kChunks;
                        if (!((seen >> row) & 1u)) st_shared_zero16(vt + (kFp8 ? swz8<HD>(row, ch) : swz<HD>(row, ch)));
                    }
                    __syncwarp();
                }
                if constexpr (kInt8) {
                    float a = ks_of[0], v = vs_of[0];
#pragma unroll
                    for (int i = 1; i < S; ++i)
                        if (sg == (uint32_t)i) {
                            a = ks_of[i];
                            v = vs_of[i];
                        }
                    st.block(kt, vt, TokenMask{seen}, lane, a, v);
                } else {
                    st.block(kt, vt, TokenMask{seen}, p.sl2, lane);
                }
                __syncwarp();
                if (lane == 0) fence_proxy_async_smem();
            }
            issue(sg);
        }
        if (dead) break;
        st.sums();
        const float inv[2] = {st.l[0] > 0.f ? 1.f / st.l[0] : 0.f, st.l[1] > 0.f ? 1.f / st.l[1] : 0.f};
        constexpr int kRun = decltype(st)::kRun;
        if (c.np == 1) {
            uint16_t* out = p.out + ((long long)c.b * p.Hq + (long long)c.h * p.G) * HD;
            st.each(lane, [&](int w, int d, const float (&v)[kRun]) {
                const int g = 2 * (lane & 3) + w;
                if (g >= p.G) return;
                if constexpr (kRun == 4)
                    *reinterpret_cast<uint2*>(out + g * HD + d) =
                        pack_bf16x4(make_float4(v[0] * inv[w], v[1] * inv[w], v[2] * inv[w], v[3] * inv[w]));
                else
                    out[g * HD + d] = f32_to_bf16(v[0] * inv[w]);
            });
        } else {
            float* part = p.part + (long long)(c.slot + c.i) * p.slot_floats;
            st.each(lane, [&](int w, int d, const float (&v)[kRun]) {
                const int g = 2 * (lane & 3) + w;
                if (g >= p.G) return;
                if constexpr (kRun == 4)
                    *reinterpret_cast<float4*>(part + g * HD + d) =
                        make_float4(v[0] * inv[w], v[1] * inv[w], v[2] * inv[w], v[3] * inv[w]);
                else
                    part[g * HD + d] = v[0] * inv[w];
            });
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int g = 2 * (lane & 3) + w;
                if (lane < 4 && g < p.G) part[p.G * HD + g] = st.l[w] > 0.f ? st.m[w] + log2f(st.l[w]) : kNegInf;
            }
            if (last_piece(p, c.slot, c.np, lane)) merge_unit<HD>(p, c.b, c.h, c.slot, c.np, lane);
        }
        c = piece(c.x + warps);
    }
    // after a wait that ran out, the copies in flight land first
    if (dead && lane == 0)
        for (; taken < issued; ++taken) {
            const uint32_t sg = taken % S;
            if ((copied >> sg) & 1u) (void)mbar_wait_bounded(full + 8 * sg, (phase >> sg) & 1u, drain_limit(p.wait_ns));
        }
}

// A value per call, never that of an earlier one in this process, nor zero: a
// random start, then a counter.
unsigned long long slide_epoch() {
    static std::atomic<unsigned long long> ctr{0};
    static const unsigned long long start = [] {
        std::random_device rd;
        return ((unsigned long long)rd() << 32) ^ (unsigned long long)rd() ^
               (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count();
    }();
    return (start + 2 * ctr.fetch_add(1)) | 1ull;
}

// Blocks per SM of the kernels (their launch bounds; shared memory holds as many).
constexpr int kSlideBlocks = 3;

mi_status check_sliding(const mi_dims* dims, int32_t window, int32_t sinks) {
    const mi_status st = check_paged_dims(dims);
    if (st != MI_OK) return st;
    if (window < 1 || sinks < 0 || (long long)dims->B * dims->Hkv > (1LL << 30)) return MI_ERR_INVALID_ARG;
    return MI_OK;
}

int slide_slots(int sms) { return kSplitPerWarp * kSlideWarps * kSlideBlocks * sms + 64; }
size_t slot_floats(const mi_dims& D) { return (size_t)(D.Hq / D.Hkv) * D.head_dim + 8; }

// Workspace: [words | partial results].
size_t slide_bytes(const mi_dims& D, int sms) { return (size_t)slide_slots(sms) * (8 + 4 * slot_floats(D)); }

template <int HD, int VAR>
cudaError_t launch_slide(int grid, cudaStream_t st, const CUtensorMap& tk, const CUtensorMap& tv, const SlideParams& p) {
    static std::mutex mu;
    static CUcontext done[256] = {};
    static_assert(SlideShape<HD, VAR>::kBlocksPerSm == kSlideBlocks, "grid");
    constexpr int smem = SlideShape<HD, VAR>::kSmem;
    if (!raise_smem(reinterpret_cast<const void*>(slide_kernel<HD, VAR>), smem, done, mu)) return cudaErrorInvalidValue;
    return launch_pdl(slide_kernel<HD, VAR>, grid, kSlideWarps * 32, smem, st, tk, tv, p);
}

mi_status attention_sliding(const mi_dims* dims, const void* q, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale, const int32_t* block_tables,
                            const int32_t* context_lens, int32_t window, int32_t sinks, float scale, void* out,
                            void* workspace, size_t workspace_bytes, int32_t* dev_err, mi_stream_t stream, int var) {
    const mi_status ds = check_sliding(dims, window, sinks);
    if (ds != MI_OK) return ds;
    const mi_dims D = *dims;
    if (!std::isfinite(scale)) return MI_ERR_INVALID_ARG;
    if (D.B == 0) return MI_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !workspace) return MI_ERR_INVALID_ARG;
    if (var != kVarMma && (!k_scale || !v_scale || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4)))
        return MI_ERR_INVALID_ARG;
    for (const void* x : {q, k_cache, v_cache, (const void*)out, (const void*)workspace})
        if (!aligned_to(x, 16)) return MI_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return MI_ERR_CUDA;
    if (workspace_bytes < slide_bytes(D, sms)) return MI_ERR_INVALID_ARG;
    const int HD = D.head_dim;
    CUtensorMap tk, tv;
    const long long rows = (long long)D.num_blocks * D.Hkv * kBlock;
    const bool maps = var == kVarMma ? make_tmap(&tk, k_cache, rows, HD) && make_tmap(&tv, v_cache, rows, HD)
                                     : make_tmap8(&tk, k_cache, rows, HD) && make_tmap8(&tv, v_cache, rows, HD);
    if (!maps) return MI_ERR_CUDA;
    SlideParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = static_cast<uint16_t*>(out);
    p.most = slide_slots(sms);
    p.words = static_cast<unsigned long long*>(workspace);
    p.part = reinterpret_cast<float*>(p.words + p.most);
    p.epoch = slide_epoch();
    p.k_scale = var == kVarFp8 ? k_scale : nullptr;
    p.v_scale = var == kVarFp8 ? v_scale : nullptr;
    p.k_amax = var == kVarInt8 ? k_scale : nullptr;
    p.v_amax = var == kVarInt8 ? v_scale : nullptr;
    p.dev_err = dev_err;
    p.B = D.B;
    p.Hq = D.Hq;
    p.Hkv = D.Hkv;
    p.G = D.Hq / D.Hkv;
    p.num_blocks = D.num_blocks;
    p.mbps = D.max_blocks_per_seq;
    p.window = window;
    p.sinks = sinks;
    p.slot_floats = (int)slot_floats(D);
    p.sl2 = scale * 1.4426950408889634f;
    // 6.8 TB/s; a warp's block takes about 0.75 us
    p.flow = (float)(2 * kBlock * HD * elem_bytes(var)) / 6.8e12f / 0.75e-6f;
    p.wait_ns = test_wait_limit_ns();
    p.withhold = test_withhold_copy() ? 1 : 0;
    const int grid = kSlideBlocks * sms;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (var == kVarMma)
        e = HD == 64 ? launch_slide<64, kVarMma>(grid, st, tk, tv, p) : launch_slide<128, kVarMma>(grid, st, tk, tv, p);
    else if (var == kVarFp8)
        e = HD == 64 ? launch_slide<64, kVarFp8>(grid, st, tk, tv, p) : launch_slide<128, kVarFp8>(grid, st, tk, tv, p);
    else
        e = HD == 64 ? launch_slide<64, kVarInt8>(grid, st, tk, tv, p) : launch_slide<128, kVarInt8>(grid, st, tk, tv, p);
    return e == cudaSuccess ? MI_OK : MI_ERR_CUDA;
}

}  // namespace
}  // namespace mi

extern "C" size_t mi_paged_sliding_workspace_bytes(const mi_dims* dims, int32_t window, int32_t sinks) {
    if (mi::check_sliding(dims, window, sinks) != MI_OK) return 0;
    const int sms = mi::sm_count();
    return sms > 0 ? mi::slide_bytes(*dims, sms) : 0;
}

extern "C" mi_status mi_paged_decode_attention_sliding(const mi_dims* dims, const void* q, const void* k_cache,
                                                       const void* v_cache, const int32_t* block_tables,
                                                       const int32_t* context_lens, int32_t window, int32_t sinks,
                                                       float scale, void* out, void* workspace, size_t workspace_bytes,
                                                       int32_t* dev_err, mi_stream_t stream) {
    return mi::attention_sliding(dims, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, window, sinks,
                                 scale, out, workspace, workspace_bytes, dev_err, stream, mi::kVarMma);
}

extern "C" mi_status mi_paged_decode_attention_sliding_fp8(const mi_dims* dims, const void* q, const void* k_cache,
                                                           const void* v_cache, const float* k_scale,
                                                           const float* v_scale, const int32_t* block_tables,
                                                           const int32_t* context_lens, int32_t window, int32_t sinks,
                                                           float scale, void* out, void* workspace,
                                                           size_t workspace_bytes, int32_t* dev_err,
                                                           mi_stream_t stream) {
    return mi::attention_sliding(dims, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, window, sinks,
                                 scale, out, workspace, workspace_bytes, dev_err, stream, mi::kVarFp8);
}

extern "C" mi_status mi_paged_decode_attention_sliding_int8(const mi_dims* dims, const void* q, const void* k_cache,
                                                            const void* v_cache, const float* k_amax,
                                                            const float* v_amax, const int32_t* block_tables,
                                                            const int32_t* context_lens, int32_t window, int32_t sinks,
                                                            float scale, void* out, void* workspace,
                                                            size_t workspace_bytes, int32_t* dev_err,
                                                            mi_stream_t stream) {
    return mi::attention_sliding(dims, q, k_cache, v_cache, k_amax, v_amax, block_tables, context_lens, window, sinks,
                                 scale, out, workspace, workspace_bytes, dev_err, stream, mi::kVarInt8);
}
