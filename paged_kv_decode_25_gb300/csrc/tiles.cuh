// 64-row tiles of bf16 rows in padded shared memory and their products on
// mma.sync, for the operators' small cases.
#pragma once

#include "common.cuh"

namespace mi {

constexpr int kTileThreads = 128;  // 4 warps
constexpr int kTileRows = 64;      // rows or keys per tile

// Padded rows: 16-byte chunks of consecutive rows fall into different banks.
template <int HD>
constexpr int kPitch = HD * 2 + 16;

// 64 rows of HD bf16 into shared memory; row(i) is the source of row i or null.
template <int HD, typename Row>
__device__ __forceinline__ void load_tile(unsigned char* tile, Row row) {
    constexpr int kChunks = HD / 8;
    for (int i = threadIdx.x; i < kTileRows * kChunks; i += kTileThreads) {
        const uint16_t* src = row(i / kChunks);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (src) v = *reinterpret_cast<const uint4*>(src + (i % kChunks) * 8);
        *reinterpret_cast<uint4*>(tile + (i / kChunks) * kPitch<HD> + (i % kChunks) * 16) = v;
    }
}

// Fragments of 16 rows x HD of a tile as the A operand of m16n8k16.
template <int HD>
__device__ __forceinline__ void load_a(uint32_t (&a)[HD / 16][4], uint32_t tile, int row0, int lane) {
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk)
        ldsm_x4(tile + (row0 + (lane & 15)) * kPitch<HD> + kk * 32 + (lane >> 4) * 16, a[kk][0], a[kk][1], a[kk][2],
                a[kk][3]);
}

// c[2][4]: products of those rows with rows col0 .. col0 + 15 of another tile.
template <int HD>
__device__ __forceinline__ void product16(float (&c)[2][4], const uint32_t (&a)[HD / 16][4], uint32_t tile, int col0,
                                          int lane) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
        uint32_t b00, b01, b10, b11;
        ldsm_x4(tile + (col0 + (lane >> 4) * 8 + (lane & 7)) * kPitch<HD> + kk * 32 + ((lane >> 3) & 1) * 16, b00, b01,
                b10, b11);
        mma_bf16_16816(c[0], a[kk][0], a[kk][1], a[kk][2], a[kk][3], b00, b01);
        mma_bf16_16816(c[1], a[kk][0], a[kk][1], a[kk][2], a[kk][3], b10, b11);
    }
}

}  // namespace mi
