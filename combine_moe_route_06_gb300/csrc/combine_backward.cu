// combine_backward.cu -- gradient of the weighted combine.
//
// out[n] = sum_j w_nj y[row(n, j)] gives, for every received pair,
//   dy[row(n, j)] = w_nj dout[n]          (bf16, one rounding)
//   dw_nj         = <y[row(n, j)], dout[n]>  (fp32 sums)
// Rows of dy that hold no pair (run padding) are set to zero.  The bound is
// HBM: every received row read and written once, dout read once.
//
// One warp per token: a 16-byte vector of dout per lane serves all of the
// token's rows, whose loads are issued together.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "trace.h"

namespace moe {

namespace {

constexpr int kCbThreads = 256;
constexpr int kCbBatch = 8;   // rows whose loads are issued together

__device__ __forceinline__ float dot_bf16x8(int4 a, int4 b, float acc)
{
    const uint32_t u[4] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w};
    const uint32_t v[4] = {(uint32_t)b.x, (uint32_t)b.y, (uint32_t)b.z, (uint32_t)b.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        acc = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), acc);
        acc = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), acc);
    }
    return acc;
}

__device__ __forceinline__ int4 scale_bf16x8(int4 a, float w)
{
    const uint32_t u[4] = {(uint32_t)a.x, (uint32_t)a.y, (uint32_t)a.z, (uint32_t)a.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(w * __uint_as_float(u[i] << 16),
                                                       w * __uint_as_float(u[i] & 0xffff0000u));
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_int4((int)r[0], (int)r[1], (int)r[2], (int)r[3]);
}

__global__ void __launch_bounds__(kCbThreads) k_combine_backward(
    const int4 *__restrict__ dout, const int4 *__restrict__ y, int y_rows,
    const int32_t *__restrict__ pair_row, const float *__restrict__ w,
    const int32_t *__restrict__ recv_pair, int64_t N, int k, int V, int4 *__restrict__ dy,
    float *__restrict__ dw, uint32_t *dev_status)
{
    pdl_wait();
    pdl_trigger();
    bool bad_row = false;
    const int lane = threadIdx.x & 31;
    const int64_t gwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t gw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    for (int64_t n = gw; n < N; n += gwarps) {
        int pr = -1;
        float wj = 0.f;
        if (lane < k) {
            pr = __ldg(pair_row + n * k + lane);
            wj = __ldg(w + n * k + lane);
            if (pr >= y_rows) {
                bad_row = true;
                pr = -1;
            }
        }
        unsigned vmask = __ballot_sync(kFull, pr >= 0);
        float mine = 0.f;             // lane j: gradient of weight j
        const int4 *g = dout + n * V;
        while (vmask) {
            int rows[kCbBatch], js[kCbBatch];
            float wb[kCbBatch], acc[kCbBatch];
#pragma unroll
            for (int b = 0; b < kCbBatch; b++) {
                const int j = vmask ? __ffs(vmask) - 1 : 0;
                js[b] = vmask ? j : -1;
                rows[b] = __shfl_sync(kFull, pr, j);
                wb[b] = __shfl_sync(kFull, wj, j);
                acc[b] = 0.f;
                vmask &= vmask - 1;
            }
            for (int v = lane; v < V; v += 32) {
                const int4 d = g[v];
                int4 r[kCbBatch];
#pragma unroll
                for (int b = 0; b < kCbBatch; b++)
                    if (js[b] >= 0) r[b] = ld_stream(y + (int64_t)rows[b] * V + v);
#pragma unroll
                for (int b = 0; b < kCbBatch; b++)
                    if (js[b] >= 0) {
                        acc[b] = dot_bf16x8(r[b], d, acc[b]);
                        st_stream(dy + (int64_t)rows[b] * V + v, scale_bf16x8(d, wb[b]));
                    }
            }
#pragma unroll
            for (int b = 0; b < kCbBatch; b++) {
                float a = acc[b];
#pragma unroll
                for (int off = 16; off; off >>= 1) a += __shfl_xor_sync(kFull, a, off);
                if (lane == js[b]) mine = a;
            }
        }
        if (lane < k) dw[n * k + lane] = mine;
    }
    if (recv_pair) {
        // rows that hold no pair: 32 rows' marks per warp step
        for (int64_t r0 = gw * 32; r0 < y_rows; r0 += gwarps * 32) {
            const bool pad = r0 + lane < y_rows && __ldg(recv_pair + r0 + lane) < 0;
            for (unsigned m = __ballot_sync(kFull, pad); m; m &= m - 1) {
                int4 *row = dy + (r0 + __ffs(m) - 1) * V;
                for (int v = lane; v < V; v += 32) st_stream(row + v, make_int4(0, 0, 0, 0));
            }
        }
    }
    if (bad_row) flag_status(dev_status, MOE_ERR_INVALID_ARG);
}

}  // namespace

cudaError_t launch_combine_backward(const uint16_t *d_out, const uint16_t *y, int y_rows,
                                    const int32_t *pair_row, const float *w,
                                    const int32_t *recv_pair, int64_t N, int k, int H,
                                    uint16_t *d_y, float *d_w, uint32_t *dev_status,
                                    cudaStream_t st)
{
    const int64_t tasks = N > (y_rows + 31) / 32 || !recv_pair ? N : (y_rows + 31) / 32;
    if (tasks == 0) return cudaSuccess;
    const int64_t want = (tasks + kCbThreads / 32 - 1) / (kCbThreads / 32);
    const int64_t fit = resident_grid((const void *)k_combine_backward, kCbThreads, 0);
    const int64_t grid = fit > 0 && want > fit ? fit : want;
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_combine_backward", st,
        err = launch_pdl(k_combine_backward, dim3((unsigned)grid), dim3(kCbThreads), 0, st,
                         (const int4 *)d_out, (const int4 *)y, y_rows, pair_row, w, recv_pair, N, k,
                         H / 8, (int4 *)d_y, d_w, dev_status));
    return err;
}

}  // namespace moe
