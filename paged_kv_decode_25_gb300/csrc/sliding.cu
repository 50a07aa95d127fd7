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
// others the warp that counts the last piece adds all of them up by their
// log-sum-exps. (A second launch for that cost 5 us a call more.)
//
// Measured, calls in a row over inputs that L2 does not hold, bytes in sight over the
// call's time: 64 requests behind windows of 1,024 (32/8 heads of 128, bf16) 48.7 us, 5.1
// TB/s, of which the stream itself runs at 7 between 6 us of plan and first copies and 4 to 5
// of last pieces; 128 behind 4,096 (28/4, e4m3) 94 us, 5.5 TB/s: no pipe is busy above 41 %
// (integer; issue 35, tensor 15), the warps wait for their own results, so one-byte blocks
// go two to a stage (on the device 92 us, 97 with one); 256 behind 128 (16/8, INT8) 27 us,
// 2.3 TB/s (24.6 on the device): 1.1 rounds of pieces of 2 to 5 double blocks, each behind
// a load of its queries (integer pipe 26 %, issue 23). A single request takes 11 us,
// latency from end to end.
#include <atomic>
#include <chrono>
#include <cmath>
#include <random>

#include "batch.cuh"
#include "common.cuh"
#include "decode_tiles.cuh"
#include "sliding.cuh"
#include "sliding_plan.cuh"
#include "tma.cuh"

namespace mi {
namespace {

template <int HD, int VAR>
struct SlideShape {
    static constexpr int kTile = Tile<HD, elem_bytes(VAR)>::kBytes;
    // blocks of a stage: what surrounds a tile (waiting, masks, the next copies, the
    // running maximum) is half of a one-byte block's instructions
    static constexpr int kBlocks = elem_bytes(VAR) == 1 ? 2 : 1;
    static constexpr int kStage = kBlocks * 2 * kTile;
    static constexpr int kStages = 16384 / kStage < 4 ? 16384 / kStage : 4;
    static constexpr int kSmem = kSlideWarps * kStages * kStage + 1024;  // slack to align the tiles
};

// Piece i of the np of (request b, head h): blocks in sight j .. j1 - 1; `slot`: the
// unit's first partial result. b < 0: no more pieces.
struct SlidePiece {
    int b, h, i, np, slot, j, j1;
};
constexpr int kPieceRing = 8;
// Units that a warp may have finished until its block adds them up. (A warp has 8
// split pieces on average at most, and of a unit's pieces one is the last; more come
// together where split units lie as far apart as there are warps.)
constexpr int kOwed = 8;

struct SlideParams {
    const uint16_t* q;             // [B][Hq][HD]
    const int32_t* block_tables;   // [B][mbps]
    const int32_t* context_lens;   // [B]
    uint16_t* out;                 // [B][Hq][HD]
    unsigned long long* words;     // [most]: at a split unit's first piece: tag | pieces done
    unsigned long long tag;        // of the call, in the high 48 bits; never zero
    float* part;                   // [most][slot_floats] normalised output [G][HD], log2-sum-exps [G]
    const float* k_scale;          // [Hkv] e4m3 caches
    const float* v_scale;
    const float* k_amax;           // [num_blocks][Hkv] INT8 caches
    const float* v_amax;
    int32_t* dev_err;
    int B, Hq, Hkv, G, num_blocks, mbps, window, sinks, most, slot_floats;
    float sl2;                     // scale * log2(e)
    float flow, alone;             // slide_flow, slide_alone
    long long wait_ns;
    int withhold;                  // failure-detection test: each warp withholds its first copy
};

__device__ __forceinline__ Sight sight_of(const SlideParams& p, int b) {
    const int n = __ldg(p.context_lens + b), cap = p.mbps * kBlock;
    return Sight(n < 0 ? 0 : (n > cap ? cap : n), p.window, p.sinks);
}

// The best of 32 cuts, chosen by every block of the launch alike.
__device__ Cut cut_units(const SlideParams& p, float warps, float blocks, float units, int largest, int hd, int lane) {
    const CutSizes sizes = {warps, blocks, units, largest, p.G * hd, p.flow, p.alone};
    CutTry c = try_cut(sizes, lane, [](float a, float b) { return __fdividef(a, b); });
    float cost = c.cost;
    int who = lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, cost, o);
        const int w = __shfl_xor_sync(0xffffffffu, who, o);
        if (x < cost || (x == cost && w < who)) {
            cost = x;
            who = w;
        }
    }
    c.step = __shfl_sync(0xffffffffu, c.step, who);
    c.tail_step = __shfl_sync(0xffffffffu, c.tail_step, who);
    c.part = __shfl_sync(0xffffffffu, c.part, who);
    return Cut(c, p.B, largest);
}

// A split unit counts its finished pieces in a word: the call's tag in the high 48
// bits, the pieces in the low 16. A word with another tag (of an earlier call, or
// whatever the workspace held) counts as zero: the first piece sets it up at its
// start, so that at the ends an addition is enough. (Counting by compare-and-swap
// alone lets one piece on per trip to L2: 54 us for a request in 22 pieces a head.)
// The last piece zeroes the word: a captured call keeps its tag.
constexpr unsigned long long kCount = 0xFFFFull;

__device__ __forceinline__ void open_count(unsigned long long* word, unsigned long long tag) {
    const unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
    if ((old & ~kCount) != tag) atomicCAS(word, old, tag);
}

// Counts a piece whose result has been written (a lane's call, the warp's results
// before a __syncwarp); whether it was the unit's last.
__device__ __forceinline__ bool last_piece(const SlideParams& p, int slot, int np) {
    unsigned long long* word = p.words + slot;
    // this warp's result before the count; the others' after it, if they are wanted
    unsigned long long old;
    asm volatile("atom.release.gpu.global.add.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
    while ((old & ~kCount) != p.tag) {
        unsigned long long seen = *reinterpret_cast<volatile unsigned long long*>(word), got;
        if ((seen & ~kCount) == p.tag) {
            asm volatile("atom.release.gpu.global.add.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
        } else {
            asm volatile("atom.release.gpu.global.cas.b64 %0, [%1], %2, %3;"
                         : "=l"(got) : "l"(word), "l"(seen), "l"(p.tag | 1ull) : "memory");
            if (got == seen) old = p.tag;
        }
    }
    const bool last = (int)(old & kCount) + 1 == np;
    if (last) {
        asm volatile("fence.acq_rel.gpu;" ::: "memory");
        *reinterpret_cast<volatile unsigned long long*>(word) = 0ull;
    }
    return last;
}

// 128 outputs of a unit, four a lane, from its np pieces in order: out = sum
// 2^(lse - M) o over the weights' sum, eight pieces' loads in flight.
template <int HD>
__device__ void merge_outputs(const SlideParams& p, int b, int h, int slot, int np, int group, int lane) {
    const int outs = p.G * HD, x = group * 128 + 4 * lane;
    if (x >= outs) return;
    const float* part = p.part + (long long)slot * p.slot_floats;
    float top = kNegInf, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0; i0 < np; i0 += 8) {
        float lse[8];
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // (past the last piece: the last one again, with no weight)
            const float* at = part + (long long)min(i0 + i, np - 1) * p.slot_floats;
            lse[i] = __ldcg(at + outs + x / HD);
            v[i] = __ldcg(reinterpret_cast<const float4*>(at + x));
        }
        float t = top;
        bool any = top != kNegInf;  // (a NaN, which fmaxf passes over, counts)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t = fmaxf(t, lse[i]);
            any |= lse[i] != kNegInf;
        }
        if (!any) continue;  // nothing in sight so far
        const float f = ex2(top - t);
        top = t;
        den *= f;
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = i0 + i < np ? ex2(lse[i] - t) : 0.f;
            den += w;
            acc.x += w * v[i].x;
            acc.y += w * v[i].y;
            acc.z += w * v[i].z;
            acc.w += w * v[i].w;
        }
    }
    const float r = den > 0.f ? 1.f / den : 0.f;
    uint16_t* out = p.out + ((long long)b * p.Hq + (long long)h * p.G) * HD + x;
    *reinterpret_cast<uint2*>(out) = pack_bf16x4(make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r));
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
__global__ void __launch_bounds__(kSlideWarps * 32, kSlideBlocks)
    slide_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const SlideParams p) {
    using Shape = SlideShape<HD, VAR>;
    constexpr int S = Shape::kStages, kTile = Shape::kTile, kThreads = kSlideWarps * 32;
    constexpr int kBlocks = Shape::kBlocks, kStage = Shape::kStage;
    constexpr bool kInt8 = VAR == kVarInt8, kFp8 = VAR == kVarFp8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long bars[kSlideWarps * S];
    __shared__ float maxima[kInt8 ? kSlideWarps * S * 2 * kBlocks : 1];  // of a stage's blocks: K's, V's
    // usual batches: blocks in sight, pieces before, those of split units; larger ones: chunks' sums
    __shared__ union {
        struct {
            int held[kFlatOneWarp], first[kFlatOneWarp + 1], first_split[kFlatOneWarp], split;
        };
        struct {
            long long sums[flat_words(kThreads)], split_sums[flat_words(kThreads)];
        };
    } plan;
    __shared__ long long red[2][kSlideWarps];
    __shared__ int red_ends[2][kSlideWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t full = smem_u32(bars) + warp * S * 8;
    const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + (uint32_t)(warp * S * kStage);
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(full + 8 * i, kInt8 ? 2 : 1);  // the tiles; the maxima
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    // ---------------------------------------------------------- the plan --
    const bool small = p.B <= kFlatOneWarp;
    long long blocks = 0, units = 0;  // (head, block)s in sight; (request, head)s with any
    int largest = 0, smallest = 0x7FFFFFFF;
    for (int b = tid; b < p.B; b += kThreads) {
        const int n = __ldg(p.context_lens + b);
        const int nb = sight_of(p, b).blocks;
        if (small) plan.held[b] = nb;
        blocks += (long long)p.Hkv * nb;
        units += nb > 0 ? p.Hkv : 0;
        largest = max(largest, nb);
        smallest = min(smallest, nb);
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
        smallest = min(smallest, __shfl_xor_sync(0xffffffffu, smallest, o));
    }
    if (lane == 0) {
        red[0][warp] = blocks;
        red[1][warp] = units;
        red_ends[0][warp] = largest;
        red_ends[1][warp] = smallest;
    }
    __syncthreads();
    blocks = units = 0;
    for (int i = 0; i < kSlideWarps; ++i) {
        blocks += red[0][i];
        units += red[1][i];
        largest = max(largest, red_ends[0][i]);
        smallest = min(smallest, red_ends[1][i]);
    }
    if (largest == 0) return;
    const int warps = gridDim.x * kSlideWarps;
    const Cut cut = cut_units(p, (float)warps, (float)blocks, (float)units, largest, HD, lane);
    auto pieces_of = [&](int b, int nb) { return cut.pieces(b, nb); };
    auto pieces = [&](int b) { return (long long)p.Hkv * pieces_of(b, sight_of(p, b).blocks); };
    auto splits = [&](int b) {
        const int np = pieces_of(b, sight_of(p, b).blocks);
        return np > 1 ? (long long)p.Hkv * np : 0LL;
    };
    const EvenCut even(cut, p.B, p.Hkv, smallest, largest);
    int total;
    bool fits = true;  // the split pieces have places (as they must, see try_cut)
    if (even.even) {
        total = even.total(p.B);
        fits = even.split(p.B) <= p.most;
    } else if (small) {
        if (warp == 0) {
            const int per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
            int v = 0, w = 0;
            for (int b = b0; b < b1; ++b) {
                const int np = pieces_of(b, plan.held[b]);
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
            if (lane == 31) {
                plan.first[p.B] = x;
                plan.split = y;
            }
            x -= v;
            y -= w;
            for (int b = b0; b < b1; ++b) {
                const int np = pieces_of(b, plan.held[b]);
                plan.first[b] = x;
                plan.first_split[b] = y;
                x += p.Hkv * np;
                y += np > 1 ? p.Hkv * np : 0;
            }
        }
        __syncthreads();
        total = plan.first[p.B];
        fits = plan.split <= p.most;
    } else {
        total = (int)flat_scan(p.B, pieces, plan.sums);
        fits = flat_scan(p.B, splits, plan.split_sums) <= p.most;
    }
    if (!fits) {
        if (tid == 0) raise_err(p.dev_err, MI_DEVERR_INTERNAL);
        return;
    }
    // ---------------------------------------------------------- the pieces --
    // The issuing side runs up to S blocks ahead, across pieces, and looks one piece
    // further: its place and first table entries (32 at a time) are there when the
    // copies reach it. The computing side finds the pieces in a ring (S + 3 at most:
    // the one computed, one for each block ahead, the one copied next, the one after).
    __shared__ SlidePiece ring_of[kSlideWarps][kPieceRing];
    static_assert(S + 3 <= kPieceRing, "pieces in flight");
    SlidePiece* pieces_ahead = ring_of[warp];
    // (neighbouring pieces on different SMs: one-byte tiles keep an SM's warps busy,
    // so all SMs get the same number of them)
    int x = warp * (int)gridDim.x + (int)blockIdx.x;  // the piece to be found next
    int found = 0, next_entry = -1;
    auto entries = [&](int b, int j, int j1) {
        return j + lane < j1 ? __ldg(p.block_tables + (long long)b * p.mbps + sight_of(p, b).column(j + lane)) : -1;
    };
    auto locate = [&](int x) {
        SlidePiece c;
        c.b = -1;
        c.np = c.j = c.j1 = 0;
        if (x < total) {
            int o, nb;
            if (even.even) {
                even.find(x, c.b, o, c.slot);
                nb = small ? plan.held[c.b] : sight_of(p, c.b).blocks;
            } else if (small) {
                int lo = 0, hi = p.B;  // first[lo] <= x < first[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (plan.first[mid] <= x) lo = mid;
                    else hi = mid;
                }
                c.b = lo;
                nb = plan.held[lo];
                o = x - plan.first[lo];
                c.slot = plan.first_split[lo];
            } else {
                long long before;
                c.b = flat_find(p.B, pieces, plan.sums, x, before);
                nb = sight_of(p, c.b).blocks;
                o = (int)(x - before);
                c.slot = (int)flat_before(p.B, splits, plan.split_sums, c.b);
            }
            c.np = pieces_of(c.b, nb);
            c.h = o / c.np;
            c.i = o - c.h * c.np;
            c.slot += c.h * c.np;
            // shares of the unit's blocks that differ by one at most
            const int share = nb / c.np, rest = nb - share * c.np;
            c.j = c.i * share + min(c.i, rest);
            c.j1 = c.j + share + (c.i < rest ? 1 : 0);
        }
        return c;
    };
    auto find = [&]() {
        const SlidePiece c = locate(x);
        if (x < total) x += warps;
        if (lane == 0) pieces_ahead[found & (kPieceRing - 1)] = c;
        ++found;
        next_entry = entries(max(c.b, 0), c.j, c.j1);
    };
    int in_b = -1, in_h = 0, in_j = 0, in_j1 = 0, entry = -1, ahead = 0;  // the piece that is copied; b < 0: none
    auto advance = [&]() {
        __syncwarp();
        const SlidePiece& c = pieces_ahead[(found - 1) & (kPieceRing - 1)];
        in_b = c.b;
        in_h = c.h;
        in_j = c.j;
        in_j1 = c.j1;
        entry = next_entry;
        ahead = 0;
        if (in_b >= 0) find();
    };
    const uint64_t policy = l2_policy_evict_first();
    find();
    advance();
    uint32_t copied = 0, phase = 0;  // bits kBlocks i ..: stage i's blocks that it holds, or will; bit i: its parity
    bool withhold = p.withhold != 0;
    auto issue = [&](uint32_t st) {
        if (in_b < 0) return;
        const int n = kBlocks == 1 ? 1 : min(kBlocks, in_j1 - in_j);
        uint32_t have = 0;
        int blk[kBlocks];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            blk[i] = __shfl_sync(0xffffffffu, entry, ahead + i);  // (`ahead` a multiple of kBlocks)
            if (i < n && blk[i] >= 0 && blk[i] < p.num_blocks) have |= 1u << i;
        }
        if (lane == 0) {
            if (have != (1u << n) - 1u) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
            if (have && !withhold) {
                const uint32_t bar = full + 8 * st;
                mbar_arrive_expect_tx(bar, (uint32_t)__popc(have) * 2 * kTile);
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    if (!((have >> i) & 1u)) continue;
                    const uint32_t dst = ring + st * kStage + i * 2 * kTile;
                    const int y = (blk[i] * p.Hkv + in_h) * (kTile / 128);
                    tma_load_2d(dst, &tmk, bar, 0, y, policy);
                    tma_load_2d(dst + kTile, &tmv, bar, 0, y, policy);
                }
                if constexpr (kInt8) {
                    // the blocks' maxima arrive on the same barrier
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i) {
                        if (!((have >> i) & 1u)) continue;
                        const uint32_t at = smem_u32(maxima + ((warp * S + st) * kBlocks + i) * 2);
                        const long long e = (long long)blk[i] * p.Hkv + in_h;
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(p.k_amax + e) : "memory");
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 4), "l"(p.v_amax + e) : "memory");
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
                }
            }
        }
        withhold = false;
        copied |= have << (kBlocks * st);
        ahead += n;
        in_j += n;
        if (in_j == in_j1) {
            advance();
        } else if (ahead == 32) {
            ahead = 0;
            entry = entries(in_b, in_j, in_j1);
        }
    };
    for (int i = 0; i < S; ++i) issue((uint32_t)i);
    uint32_t sg = 0;  // the stage whose block comes next
    bool dead = false;
    typename TileOf<HD, VAR>::T st;
    // The units whose last piece was one of this warp's, to be added up at the end (sums
    // among the tiles' registers spilled, which cost the e4m3 tiles a third of their
    // rate); pieces past the first kOwed of those are counted there, too.
    __shared__ int4 owed[kSlideWarps][kOwed];  // {request, head, first partial result, pieces}
    __shared__ int owed_count[kSlideWarps];
    int owes = 0, counted = 0;
    for (int done = 0;; ++done) {
        __syncwarp();
        const SlidePiece& c = pieces_ahead[done & (kPieceRing - 1)];
        if (dead || c.b < 0) break;
        const Sight sight = sight_of(p, c.b);
        st.begin_unit(p, c.b, c.h, lane);
        if (c.np > 1 && c.i == 0 && lane == 0) open_count(p.words + c.slot, p.tag);
        const int j1 = c.j1;
        for (int j = c.j; j < j1; j += kBlocks) {
            const uint32_t have = (copied >> (kBlocks * sg)) & ((1u << kBlocks) - 1u);
            if (have) {
                if (!wait_warp(full + 8 * sg, (phase >> sg) & 1u, p.wait_ns)) {
                    if (lane == 0) raise_err(p.dev_err, MI_DEVERR_TIMEOUT);
                    dead = true;
                    break;
                }
                phase ^= 1u << sg;
                copied &= ~(have << (kBlocks * sg));
                const uint32_t kt = ring + sg * kStage, vt = kt + kTile;
                uint32_t seen = 0;
#pragma unroll
                for (int i = 0; i < kBlocks; ++i)
                    if ((have >> i) & 1u) seen |= sight.mask(sight.column(j + i)) << (kBlock * i);
                if (!kInt8 && seen != (kBlocks == 2 ? 0xFFFFFFFFu : 0xFFFFu)) {
                    // rows out of sight may hold any bits: zero V there (INT8 codes are always finite)
                    constexpr int kChunks = HD * elem_bytes(VAR) / 16;
                    for (int i = lane; i < kBlocks * kBlock * kChunks; i += 32) {
                        const int at = i / kChunks, row = at % kBlock, ch = i % kChunks;
                        const uint32_t tile = vt + at / kBlock * 2 * kTile;
                        if (!((seen >> at) & 1u)) st_shared_zero16(tile + (kFp8 ? swz8<HD>(row, ch) : swz<HD>(row, ch)));
                    }
                    __syncwarp();
                }
                if constexpr (kInt8) {
                    const float* m = maxima + (warp * S + sg) * kBlocks * 2;
                    // (an absent block's maxima are an earlier one's)
                    st.pair(kt, vt, 2 * kTile, TokenMask{seen}, lane, have & 1u ? m[0] : 0.f, have & 2u ? m[2] : 0.f,
                            have & 1u ? m[1] : 0.f, have & 2u ? m[3] : 0.f);
                } else if constexpr (kFp8) {
                    st.pair(kt, vt, 2 * kTile, TokenMask{seen}, lane);
                } else {
                    st.block(kt, vt, TokenMask{seen}, p.sl2, lane);
                }
                __syncwarp();
                if (lane == 0) fence_proxy_async_smem();
            }
            issue(sg);
            sg = sg + 1 == S ? 0 : sg + 1;
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
                if (lane < 4 && g < p.G) part[p.G * HD + g] = st.l[w] == 0.f ? kNegInf : st.m[w] + log2f(st.l[w]);
            }
            __syncwarp();
            if (counted == done && owes < kOwed) {
                int last = 0;
                if (lane == 0 && last_piece(p, c.slot, c.np)) {
                    owed[warp][owes] = make_int4(c.b, c.h, c.slot, c.np);
                    last = 1;
                }
                owes += __shfl_sync(0xffffffffu, last, 0);
                ++counted;
            }
        }
        counted += c.np == 1 && counted == done;
    }
    if (dead && lane == 0)  // the copies in flight land first
        for (int i = 0; i < S; ++i)
            if ((copied >> (kBlocks * i)) & ((1u << kBlocks) - 1u)) (void)mbar_wait_bounded(full + 8 * i, (phase >> i) & 1u, drain_limit(p.wait_ns));
    if (even.n0 == 1 && even.n1 == 1) return;  // no unit is split
    // All of the block's warps add up what they owe. (One warp a unit took 12 us for two
    // units of 7 pieces and 7 heads. Counting all pieces only here left most units to
    // the blocks that end last: 185 us instead of 98 with 21 pieces a unit.)
    const int groups = (p.G * HD + 127) / 128;
    if (lane == 0) owed_count[warp] = owes;
    const int own = (total - (warp * (int)gridDim.x + (int)blockIdx.x) + warps - 1) / warps;  // this warp's pieces
    const bool more = __syncthreads_or(!dead && counted < own) != 0;
#pragma unroll 1
    for (int w = 0; w < kSlideWarps; ++w)
#pragma unroll 1
        for (int q = (warp + w) % kSlideWarps; q < owed_count[w] * groups; q += kSlideWarps) {
            const int4 u = owed[w][q / groups];
            merge_outputs<HD>(p, u.x, u.y, u.z, u.w, q % groups, lane);
        }
    if (!more) return;
    __shared__ int4 whole_units[kSlideWarps * 32];
    __shared__ int whole_count;
#pragma unroll 1
    for (int k0 = 0; k0 < (total + warps - 1) / warps; k0 += 32) {
        if (tid == 0) whole_count = 0;
        __syncthreads();
        const int k = k0 + lane;
        if (!dead && k >= counted && k < own) {
            const SlidePiece c = locate(warp * (int)gridDim.x + (int)blockIdx.x + k * warps);
            if (c.np > 1 && last_piece(p, c.slot, c.np)) whole_units[atomicAdd(&whole_count, 1)] = make_int4(c.b, c.h, c.slot, c.np);
        }
        __syncthreads();
#pragma unroll 1
        for (int q = warp; q < whole_count * groups; q += kSlideWarps) {
            const int4 u = whole_units[q / groups];
            merge_outputs<HD>(p, u.x, u.y, u.z, u.w, q % groups, lane);
        }
        __syncthreads();
    }
}

// A value per call, never that of an earlier one in this process, nor zero: a
// random start, then a counter.
unsigned long long slide_epoch() {
    static std::atomic<unsigned long long> ctr{0};
    static const unsigned long long start = [] {
        unsigned long long x = (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count();
        try {  // (no exception leaves a C entry)
            std::random_device rd;
            x ^= ((unsigned long long)rd() << 32) ^ (unsigned long long)rd();
        } catch (...) {
        }
        return x;
    }();
    return (start + 2 * ctr.fetch_add(1)) | 1ull;
}

mi_status check_sliding(const mi_dims* dims, int32_t window, int32_t sinks) {
    const mi_status st = check_paged_dims(dims);
    if (st != MI_OK) return st;
    if (window < 1 || sinks < 0 || (long long)dims->B * dims->Hkv > (1LL << 30)) return MI_ERR_INVALID_ARG;
    return MI_OK;
}

size_t slot_floats(const mi_dims& D) { return (size_t)(D.Hq / D.Hkv) * D.head_dim + 8; }

// Workspace: [words | partial results].
size_t slide_bytes(const mi_dims& D, int sms) { return (size_t)slide_slots(sms) * (8 + 4 * slot_floats(D)); }

template <int HD, int VAR>
cudaError_t launch_slide(int sms, cudaStream_t st, const CUtensorMap& tk, const CUtensorMap& tv, const SlideParams& p) {
    static std::mutex mu;
    static CUcontext done[256] = {};
    constexpr int smem = SlideShape<HD, VAR>::kSmem;
    if (!raise_smem(reinterpret_cast<const void*>(slide_kernel<HD, VAR>), smem, done, mu)) return cudaErrorInvalidValue;
    return launch_pdl(slide_kernel<HD, VAR>, kSlideBlocks * sms, kSlideWarps * 32, smem, st, tk, tv, p);
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
    p.tag = slide_epoch() << 16;
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
    p.flow = slide_flow(HD, elem_bytes(var));
    p.alone = slide_alone(elem_bytes(var));
    p.wait_ns = test_wait_limit_ns();
    p.withhold = test_withhold_copy() ? 1 : 0;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (var == kVarMma)
        e = HD == 64 ? launch_slide<64, kVarMma>(sms, st, tk, tv, p) : launch_slide<128, kVarMma>(sms, st, tk, tv, p);
    else if (var == kVarFp8)
        e = HD == 64 ? launch_slide<64, kVarFp8>(sms, st, tk, tv, p) : launch_slide<128, kVarFp8>(sms, st, tk, tv, p);
    else
        e = HD == 64 ? launch_slide<64, kVarInt8>(sms, st, tk, tv, p) : launch_slide<128, kVarInt8>(sms, st, tk, tv, p);
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
