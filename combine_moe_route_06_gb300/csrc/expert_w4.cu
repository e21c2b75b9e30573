// expert_w4.cu -- the experts' products with 4-bit weights.
//
// y[r] = factor[e] * (a[r] . W_e^T) for the rows r of expert e's run, W_e of
// E2M1 codes with one E4M3 scale per 16 columns; gated: W_e = [gate; up] and
// y[r] = silu(a[r] . gate^T) * (a[r] . up^T).  The layout and the decoding of
// the weights are in w4.cuh.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "trace.h"
#include "w4.cuh"

namespace moe {

namespace {

constexpr int kPackThreads = 256;

// One thread per 16-byte piece of a block: 32 codes and their two scales.
__global__ void __launch_bounds__(kPackThreads) k_w4_pack(const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, int E,
                                                          int N, int K, bool gated,
                                                          uint8_t *__restrict__ out)
{
    pdl_wait();
    pdl_trigger();
    const int tiles = w4_tiles(N, gated), chunks = w4_chunks(K);
    const int64_t pieces = (int64_t)E * tiles * chunks * (kW4Tile * 4);
    const int rows = gated ? 2 * N : N;
    for (int64_t at = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; at < pieces;
         at += (int64_t)gridDim.x * kPackThreads) {
        // the four pieces of a row are neighbours, so a warp reads whole 64-byte spans
        const int j = (int)(at & 3), i = (int)(at >> 2) & (kW4Tile - 1);
        const int64_t block = at / (kW4Tile * 4);
        const int c = (int)(block % chunks);
        const int t = (int)(block / chunks % tiles);
        const int e = (int)(block / chunks / tiles);
        const int n = w4_source_row(t, i, N, gated);
        const int k0 = c * kW4Chunk + j * 32;
        uint2 q[2] = {make_uint2(0, 0), make_uint2(0, 0)};
        uint32_t s[2] = {0, 0};
        if (n >= 0) {
            const int64_t row = (int64_t)e * rows + n;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (k0 + 16 * h < K) {      // K is a multiple of 16: a whole group or nothing
                    q[h] = *(const uint2 *)(codes + row * (K / 2) + (k0 + 16 * h) / 2);
                    s[h] = scales[row * (K / 16) + k0 / 16 + h];
                }
            }
        }
        uint8_t *dst = out + block * kW4BlockBytes;
        *(uint4 *)(dst + (j * kW4Tile + i) * 16) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
        *(uint16_t *)(dst + kW4CodeBytes + i * 8 + j * 2) = (uint16_t)(s[0] | (s[1] << 8));
    }
}

constexpr int kRowsAtOnce = 8;

// One CTA per (expert, tile), one thread per row of the tile, eight rows of `a`
// at a time.
__global__ void __launch_bounds__(kW4Tile) k_expert_w4(
    const __nv_bfloat16 *__restrict__ a, int a_rows, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ counts, int block_rows, const uint8_t *__restrict__ w4,
    const float *__restrict__ factor, int N, int K, bool gated, __nv_bfloat16 *__restrict__ y,
    uint32_t *dev_status)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float up[kRowsAtOnce][kW4Tile / 2];
    const int t = blockIdx.x, e = blockIdx.y, i = threadIdx.x;
    const int tiles = w4_tiles(N, gated), chunks = w4_chunks(K);
    int start, count;
    bool bad = false;
    expert_rows(offsets, counts, block_rows, a_rows, e, start, count, bad);
    if (bad && t == 0 && i == 0) flag_status(dev_status, MOE_ERR_INVALID_ARG);
    const uint8_t *w = w4 + ((int64_t)e * tiles + t) * chunks * (int64_t)kW4BlockBytes;
    const float f = factor[e];
    for (int r0 = 0; r0 < count; r0 += kRowsAtOnce) {
        const int nr = count - r0 < kRowsAtOnce ? count - r0 : kRowsAtOnce;
        float acc[kRowsAtOnce] = {};
        for (int c = 0; c < chunks; c++) {
            const uint8_t *block = w + (int64_t)c * kW4BlockBytes;
            const uint2 sc = *(const uint2 *)(block + kW4CodeBytes + i * 8);
            for (int j = 0; j < 4; j++) {
                const uint4 q = *(const uint4 *)(block + (j * kW4Tile + i) * 16);
                const uint32_t word[4] = {q.x, q.y, q.z, q.w};
                const uint32_t s2 = e4m3x2_to_half2((j < 2 ? sc.x : sc.y) >> (16 * (j & 1)));
                const float2 s = __half22float2(*(const __half2 *)&s2);
                const int k0 = c * kW4Chunk + j * 32;
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    if (k0 + 8 * v >= K) continue;
                    uint32_t h[4];
                    e2m1x8_to_half2(word[v], h);
                    float x[8];
#pragma unroll
                    for (int p = 0; p < 4; p++) {
                        const float2 q2 = __half22float2(*(const __half2 *)&h[p]);
                        x[2 * p] = q2.x * (v < 2 ? s.x : s.y);
                        x[2 * p + 1] = q2.y * (v < 2 ? s.x : s.y);
                    }
                    for (int r = 0; r < nr; r++) {
                        const __nv_bfloat16 *src = a + (int64_t)(start + r0 + r) * K + k0 + 8 * v;
#pragma unroll
                        for (int p = 0; p < 8; p++)
                            acc[r] = fmaf(__bfloat162float(src[p]), x[p], acc[r]);
                    }
                }
            }
        }
        const int per = w4_outputs_per_tile(gated);
        const int n = t * per + i % per;
        if (gated) {
            __syncthreads();
            if (i >= per)
                for (int r = 0; r < nr; r++) up[r][i - per] = acc[r] * f;
            __syncthreads();
        }
        if (i < per && n < N)
            for (int r = 0; r < nr; r++) {
                float v = acc[r] * f;
                if (gated) v = v / (1.f + expf(-v)) * up[r][i];
                y[(int64_t)(start + r0 + r) * N + n] = __float2bfloat16_rn(v);
            }
    }
}

}  // namespace

size_t w4_bytes(int E, int N, int K, bool gated)
{
    return (size_t)E * w4_tiles(N, gated) * w4_chunks(K) * kW4BlockBytes;
}

cudaError_t launch_w4_pack(const uint8_t *codes, const uint8_t *scales, int E, int N, int K,
                           bool gated, uint8_t *w4, cudaStream_t st)
{
    const int64_t pieces = (int64_t)E * w4_tiles(N, gated) * w4_chunks(K) * (kW4Tile * 4);
    const int64_t want = (pieces + kPackThreads - 1) / kPackThreads;
    const int64_t fit = resident_grid((const void *)k_w4_pack, kPackThreads, 0);
    const int64_t grid = fit > 0 && want > fit ? fit : want;
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_w4_pack", st,
        err = launch_pdl(k_w4_pack, dim3((unsigned)grid), dim3(kPackThreads), 0, st, codes, scales,
                         E, N, K, gated, w4));
    return err;
}

size_t expert_w4_ws_bytes(int a_rows, int E, int N, int K)
{
    return 256;
}

cudaError_t launch_expert_w4(const uint16_t *a, int a_rows, const int32_t *offsets,
                             const int32_t *counts, int block_rows, const uint8_t *w4,
                             const float *factor, int E, int N, int K, bool gated, uint16_t *y,
                             void *ws, uint32_t *dev_status, cudaStream_t st)
{
    if (a_rows == 0) return cudaSuccess;
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_expert_w4", st,
        err = launch_pdl(k_expert_w4, dim3(w4_tiles(N, gated), E), dim3(kW4Tile), 0, st,
                         (const __nv_bfloat16 *)a, a_rows, offsets, counts, block_rows, w4, factor,
                         N, K, gated, (__nv_bfloat16 *)y, dev_status));
    return err;
}

}  // namespace moe
