// Shared pieces of the kernels that walk a batch of requests as one flat list
// of work items, and the host-side checks of their entry points.
#pragma once

#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "tma.cuh"

namespace mi {

// ------------------------------------------------------------- flat items --
//
// Entry b of B contributes count(b) items (a count never depends on anything
// but device data that stays fixed during the launch), laid end to end in the
// order of b. Every block scans the counts itself, which is less than a launch
// that would write the list: the entries are cut into equal chunks, and sums[t]
// holds the items before chunk t, sums[chunks] the total. Up to 512 entries one
// warp does it (32 chunks, one barrier: the usual batch, where three barriers of
// a wide block were most of the plan's time); larger batches take the whole
// block, a chunk per thread.

constexpr int kFlatWarps = 32;
constexpr int kFlatOneWarp = 512;
__host__ __device__ constexpr int flat_words(int threads) { return threads + 1 + kFlatWarps; }

__device__ __forceinline__ int flat_chunks(int B) { return B <= kFlatOneWarp ? 32 : (int)blockDim.x; }

// Ends with a barrier; the caller makes sure nobody still reads `sums`.
template <typename Count>
__device__ long long flat_scan(int B, Count count, long long* sums) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int chunks = flat_chunks(B), per = (B + chunks - 1) / chunks;
    const bool one = B <= kFlatOneWarp;
    long long v = 0, x = 0;
    if (!one || wid == 0) {
        const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
        for (int b = b0; b < b1; ++b) v += count(b);
        x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
    }
    if (one) {
        if (wid == 0) {
            sums[lane] = x - v;
            if (lane == 31) sums[32] = x;
        }
        __syncthreads();
        return sums[32];
    }
    const int nt = blockDim.x, nw = (nt + 31) >> 5;
    long long* wsum = sums + nt + 1;
    if (lane == 31) wsum[wid] = x;
    __syncthreads();
    if (wid == 0) {
        long long t = lane < nw ? wsum[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        if (lane < nw) wsum[lane] = t;
    }
    __syncthreads();
    const long long before = (wid ? wsum[wid - 1] : 0) + x - v;
    sums[tid] = before;
    if (tid == nt - 1) sums[nt] = before + v;
    __syncthreads();
    return sums[nt];
}

// The entry that holds item x (0 <= x < total), and the items before it in
// `first`. Reads `sums` only, so any thread may call it at any time.
template <typename Count>
__device__ int flat_find(int B, Count count, const long long* sums, long long x, long long& first) {
    const int chunks = flat_chunks(B), per = (B + chunks - 1) / chunks;
    int lo = 0, hi = chunks;  // sums[lo] <= x < sums[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid;
    }
    int b = lo * per;
    long long acc = sums[lo];
    for (;;) {
        const long long c = count(b);
        if (x < acc + c) break;
        acc += c;
        ++b;
    }
    first = acc;
    return b;
}

// The items before entry b.
template <typename Count>
__device__ long long flat_before(int B, Count count, const long long* sums, int b) {
    const int chunks = flat_chunks(B), per = (B + chunks - 1) / chunks;
    long long acc = sums[b / per];
    for (int c = b / per * per; c < b; ++c) acc += count(c);
    return acc;
}

// Whether starts[0 .. count] ascends within [0, limit]; the same answer in
// every thread of the block (a barrier). Ranges that ascend never overlap.
__device__ inline bool starts_ascend(const int32_t* starts, int count, int limit) {
    bool ok = true;
    for (int i = threadIdx.x; i <= count; i += blockDim.x) {
        const int s = __ldg(starts + i);
        ok &= s >= 0 && s <= limit && (i == 0 || __ldg(starts + i - 1) <= s);
    }
    return __syncthreads_and(ok) != 0;
}

// ------------------------------------------------------------- host checks --

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool overlaps(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// Blocks of the longest table: token indices of a work item that begins in the
// context (up to 1,024 tokens) stay within 32 bits.
constexpr int kLongestTable = (1 << 27) - 128;

// The dims the cache operators accept (B up to 65535).
inline mi_status check_paged_dims(const mi_dims* dims) {
    if (!dims) return MI_ERR_INVALID_ARG;
    const mi_dims& D = *dims;
    if (D.B < 0 || D.B > 65535 || D.Hq < 1 || D.Hkv < 1 || D.num_blocks < 1 || D.max_blocks_per_seq < 1)
        return MI_ERR_INVALID_ARG;
    if (D.block_size != kBlock || (D.head_dim != 64 && D.head_dim != 128) || D.Hq % D.Hkv != 0 || D.Hq / D.Hkv > 8)
        return MI_ERR_UNSUPPORTED;
    if ((long long)D.num_blocks * D.Hkv * kBlock * (D.head_dim / 64) > 0x7FFFFFFFLL) return MI_ERR_INVALID_ARG;
    if (D.max_blocks_per_seq > kLongestTable) return MI_ERR_INVALID_ARG;
    return MI_OK;
}

inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

// Raises a kernel's dynamic shared-memory limit once per device context
// (`done` and `mu` are the kernel's own).
inline bool raise_smem(const void* fn, int bytes, CUcontext (&done)[256], std::mutex& mu) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lk(mu);
    const CUcontext ctx = current_context();
    if (dev >= 0 && dev < 256 && ctx && done[dev] == ctx) return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (dev >= 0 && dev < 256) done[dev] = current_context();
    return true;
}

}  // namespace mi
