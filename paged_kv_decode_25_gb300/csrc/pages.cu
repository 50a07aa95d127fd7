// mi_kv_copy_planes: one list of page moves made in every plane (each layer's K,
// V, scores, maxima) by one launch: forks' last pages, compaction. A launch per
// layer, as mi_kv_copy_blocks takes, costs more than the copies of a fork do.
//
// Bound by the bytes, once in and once out. The work is cut into items of up to
// kItemBytes: rows of a plane longer than that in pieces, several shorter rows to
// an item. A block takes one item and has all of its loads in flight before it
// stores; blocks in the order of the planes, so that neighbours work on one plane.
//
// Measured: 1,300 pages of 4 layers (8 heads of 128, bf16; 681 MB moved) 101 us, 6.7 TB/s, a
// copy's rate; 8 pages of 36 layers 6.8 us on the device (38 MB, partly from L2).
#include "batch.cuh"
#include "common.cuh"

namespace mi {
namespace {

constexpr int kPageThreads = 256;
constexpr int kPageUnroll = 8;
constexpr int kItemBytes = kPageThreads * kPageUnroll * 16;
// Planes of one launch (its arguments stay below 4 KB); more take further launches.
constexpr int kLaunchPlanes = 144;

struct Plane {
    uint8_t* base;
    long long row_bytes;
    int rows, first;  // rows of the plane; its first item
};

struct PageParams {
    const int32_t* src_ids;
    const int32_t* dst_ids;
    int32_t* dev_err;
    int n, planes, items;
    Plane plane[kLaunchPlanes];
};
static_assert(sizeof(PageParams) <= 4096 - 16, "kernel arguments");

// Rows of an item, or pieces of a row.
__host__ __device__ inline int rows_per_item(long long row_bytes) {
    return row_bytes >= kItemBytes ? 1 : (int)(kItemBytes / row_bytes);
}
__host__ __device__ inline long long pieces_per_row(long long row_bytes) {
    return (row_bytes + kItemBytes - 1) / kItemBytes;
}

// Units of `U` of the item's rows i0 .. i1 - 1, bytes `from` .. `from + len` of each.
template <typename U>
__device__ __forceinline__ void copy_item(const PageParams& p, const Plane& pl, int i0, int i1, long long from, int len) {
    const int units = len / (int)sizeof(U), total = units * (i1 - i0);
    for (int base = 0; base < total; base += kPageThreads * kPageUnroll) {
        U v[kPageUnroll];
        long long to[kPageUnroll];  // byte offset in the plane, -1: nothing
#pragma unroll
        for (int u = 0; u < kPageUnroll; ++u) {
            const int x = base + u * kPageThreads + threadIdx.x;
            to[u] = -1;
            if (x >= total) continue;
            const int i = i1 - i0 == 1 ? 0 : x / units;
            const int s = __ldg(p.src_ids + i0 + i), d = __ldg(p.dst_ids + i0 + i);
            if (s < 0 || s >= pl.rows || d < 0 || d >= pl.rows) {
                if (x == i * units) raise_err(p.dev_err, MI_DEVERR_BAD_BLOCK);
                continue;
            }
            const long long off = from + (long long)(x - i * units) * (int)sizeof(U);
            v[u] = *reinterpret_cast<const U*>(pl.base + s * pl.row_bytes + off);
            to[u] = d * pl.row_bytes + off;
        }
#pragma unroll
        for (int u = 0; u < kPageUnroll; ++u)
            if (to[u] >= 0) *reinterpret_cast<U*>(pl.base + to[u]) = v[u];
    }
}

__global__ void __launch_bounds__(kPageThreads) copy_planes_kernel(const __grid_constant__ PageParams p) {
    pdl_wait();
    pdl_trigger();
    const int item = blockIdx.x;
    int lo = 0, hi = p.planes;  // plane[lo].first <= item < plane[hi].first
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.plane[mid].first <= item) lo = mid;
        else hi = mid;
    }
    const Plane& pl = p.plane[lo];
    const int x = item - pl.first;
    const int per = rows_per_item(pl.row_bytes), pieces = (int)pieces_per_row(pl.row_bytes);
    const int i0 = x / pieces * per, i1 = i0 + min(per, p.n - i0);  // (n may be near 2^31)
    const long long from = (long long)(x % pieces) * kItemBytes;
    const int len = (int)min((long long)kItemBytes, pl.row_bytes - from);
    if (((reinterpret_cast<uintptr_t>(pl.base) | (uintptr_t)pl.row_bytes) & 15u) == 0)
        copy_item<uint4>(p, pl, i0, i1, from, len);
    else
        copy_item<uint32_t>(p, pl, i0, i1, from, len);
}

}  // namespace
}  // namespace mi

extern "C" mi_status mi_kv_copy_planes(const mi_kv_plane* planes, int32_t num_planes, const int32_t* src_ids,
                                       const int32_t* dst_ids, int32_t n, int32_t* dev_err, mi_stream_t stream) {
    using namespace mi;
    if (num_planes < 0 || n < 0 || (num_planes > 0 && !planes)) return MI_ERR_INVALID_ARG;
    for (int i = 0; i < num_planes; ++i) {
        const mi_kv_plane& pl = planes[i];
        if (!pl.base || !aligned_to(pl.base, 4) || pl.rows < 1 || pl.rows > 0x7FFFFFFFLL || pl.row_bytes < 4 ||
            pl.row_bytes % 4 != 0 || pl.row_bytes > (1LL << 40) / pl.rows)
            return MI_ERR_INVALID_ARG;
        if (n > 0 && ((n - 1LL) / rows_per_item(pl.row_bytes) + 1) > 0x7FFFFFFFLL / pieces_per_row(pl.row_bytes))
            return MI_ERR_INVALID_ARG;
    }
    if (n == 0 || num_planes == 0) return MI_OK;
    if (!src_ids || !dst_ids || !aligned_to(src_ids, 4) || !aligned_to(dst_ids, 4)) return MI_ERR_INVALID_ARG;
    PageParams p;
    p.src_ids = src_ids;
    p.dst_ids = dst_ids;
    p.dev_err = dev_err;
    p.n = n;
    p.planes = 0;
    long long items = 0;
    auto launch = [&] {
        p.items = (int)items;
        return launch_pdl(copy_planes_kernel, p.items, kPageThreads, 0, (cudaStream_t)stream, p);
    };
    for (int i = 0; i < num_planes; ++i) {
        const mi_kv_plane& pl = planes[i];
        const long long add = ((n - 1LL) / rows_per_item(pl.row_bytes) + 1) * pieces_per_row(pl.row_bytes);
        if (p.planes == kLaunchPlanes || items + add > 0x7FFFFFFFLL) {
            if (launch() != cudaSuccess) return MI_ERR_CUDA;
            p.planes = 0;
            items = 0;
        }
        p.plane[p.planes++] = Plane{static_cast<uint8_t*>(pl.base), pl.row_bytes, (int)pl.rows, (int)items};
        items += add;
    }
    return launch() == cudaSuccess ? MI_OK : MI_ERR_CUDA;
}
