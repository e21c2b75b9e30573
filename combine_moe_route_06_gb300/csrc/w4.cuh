// w4.cuh -- the 4-bit expert weights: their layout in memory and their decoding.
//
// A weight is E2M1 code x E4M3 scale of its group of 16 along K x the expert's
// fp32 factor.  code * scale has at most 6 significant bits and lies in
// [2^-10, 2688] or is 0, so it is exact in fp16 (and normal there).
//
// Packed form: blocks of 128 rows x 128 columns, 9,216 bytes each, so a block
// is one bulk copy and any row count or K is padded with zero codes.  A tile is
// one or two blocks of rows that share their columns of the other operand:
//   gated weights [gate; up]: 128 gate rows and the same 128 up rows, so that the
//     two factors of an output meet in one lane;
//   else two row blocks where their number is even, one where it is odd.
//   block h (expert e, tile t, column chunk c) at
//     (((e*tiles + t)*chunks + c)*blocks + h) * 9216
//   codes : [4][128 rows][16 bytes], piece j of a row = its columns 128c+32j .. +31,
//           first value of a byte in the low nibble
//   scales: [128 rows][8 bytes] from byte 8192 on
// Lanes that own consecutive rows read consecutive 16-byte pieces of shared memory.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

constexpr int kW4Tile = 128;                                   // rows of a block
constexpr int kW4Chunk = 128;                                  // columns of a block
constexpr int kW4CodeBytes = kW4Tile * kW4Chunk / 2;           // 8192
constexpr int kW4BlockBytes = kW4CodeBytes + kW4Tile * kW4Chunk / 16;   // 9216

// Row blocks per tile, outputs per tile, tiles and column chunks of a weight.
__host__ __device__ __forceinline__ int w4_blocks(int N, bool gated)
{
    return gated || (N + kW4Tile - 1) / kW4Tile % 2 == 0 ? 2 : 1;
}
__host__ __device__ __forceinline__ int w4_outputs(int N, bool gated)
{
    return gated ? kW4Tile : kW4Tile * w4_blocks(N, gated);
}
__host__ __device__ __forceinline__ int w4_tiles(int N, bool gated)
{
    return (N + w4_outputs(N, gated) - 1) / w4_outputs(N, gated);
}
__host__ __device__ __forceinline__ int w4_chunks(int K) { return (K + kW4Chunk - 1) / kW4Chunk; }

// Output that row i of block h of tile t belongs to (N or more: padding).
__host__ __device__ __forceinline__ int w4_output(int t, int h, int i, int N, bool gated)
{
    return gated ? t * kW4Tile + i : (t * w4_blocks(N, gated) + h) * kW4Tile + i;
}

// Eight codes (one 32-bit word, first value in the low nibble) to fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two E4M3 scales (low byte first) to an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The rows of expert e: [start, start + count) of a_rows rows, from run offsets
// or from a count per block of block_rows rows.  Device data that would leave
// the buffer is cut to it; `bad` tells.
__device__ __forceinline__ void expert_rows(const int32_t *offsets, const int32_t *counts,
                                            int block_rows, int a_rows, int e, int &start,
                                            int &count, bool &bad)
{
    int64_t s, c;
    if (offsets) {
        s = __ldg(offsets + e);
        c = (int64_t)__ldg(offsets + e + 1) - s;
    } else {
        s = (int64_t)e * block_rows;
        c = __ldg(counts + e);
        if (c > block_rows) {
            c = block_rows;
            bad = true;
        }
    }
    if (s < 0 || c < 0 || s > a_rows) {
        s = c = 0;
        bad = true;
    } else if (s + c > a_rows) {
        c = a_rows - s;
        bad = true;
    }
    start = (int)s;
    count = (int)c;
}

}  // namespace moe
