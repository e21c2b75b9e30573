// combine_backward.cu -- gradient of the weighted combine.
//
// out[n] = sum_j w_nj y[row(n, j)] gives, for every received pair,
//   dy[row(n, j)] = w_nj dout[n]          (bf16, one rounding)
//   dw_nj         = <y[row(n, j)], dout[n]>  (fp32 sums)
// Rows of dy that hold no pair (run padding) are set to zero.  The bound is
// HBM: every received row read and written once, dout read once (4,096 tokens x 6 rows
// of 5,120: 92.7 us, 5.9 TB/s, 0.87 of a plain copy's rate).
//
// One warp per token, or with few tokens one CTA, whose warps take the row's
// columns in turn: a 16-byte vector of dout per lane serves all of the token's
// rows, and nine to twelve vectors are in flight per lane (of dout and eight rows,
// or of two rows at four columns).
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "trace.h"

namespace moe {

namespace {

constexpr int kCbThreads = 256;
constexpr int kCbWarps = kCbThreads / 32;
constexpr int kCbCtas = 2;    // CTAs per SM: 128 registers a thread
// Rows of a token taken at once, where the buffer has more than two rows a token or not
// (how many of them are in use only the device knows).  4,096 tokens x 6 rows of 5,120: 92.9 us at eight, 102.7 at two; 16,384
// tokens x one row of 2,048 (of 8 picks): 37.4 us at two, 59.7 at eight (34.0 at two
// since warps take tokens as they come free).  A buffer much larger than its rows takes the
// form for many and has every unused row set to zero: the same tokens take 127 us in one of
// 131,072 rows.
constexpr int kManyRows = 8, kFewRows = 2;

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

template <int ROWS>
constexpr int kUnroll = ROWS > 4 ? 1 : ROWS > 2 ? 2 : 4;

// ROWS of the token's rows (-1: none), vectors first, first + step, ... of V:
// writes their gradients and adds their products with dout to acc.
template <int ROWS>
__device__ __forceinline__ void rows_backward(const int4 *g, const int4 *y, int4 *dy, int V,
                                              int first, int step, const int (&rows)[ROWS],
                                              const float (&w)[ROWS],
                                              float (&acc)[ROWS])
{
    constexpr int U = kUnroll<ROWS>;
#pragma unroll 1
    for (int v0 = first; v0 < V; v0 += U * step) {
        int4 d[U], r[U][ROWS];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int v = v0 + u * step;
            if (v < V) d[u] = ld_stream(g + v);
#pragma unroll
            for (int b = 0; b < ROWS; b++)
                if (v < V && rows[b] >= 0) r[u][b] = ld_stream(y + (int64_t)rows[b] * V + v);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int v = v0 + u * step;
#pragma unroll
            for (int b = 0; b < ROWS; b++)
                if (v < V && rows[b] >= 0) {
                    acc[b] = dot_bf16x8(r[u][b], d[u], acc[b]);
                    st_stream(dy + (int64_t)rows[b] * V + v, scale_bf16x8(d[u], w[b]));
                }
        }
    }
}

// The next ROWS received rows of the token (bits of vmask); lane j of `mine` gets
// the warp's sum of row j.
template <int ROWS>
__device__ __forceinline__ void batch_backward(const int4 *g, const int4 *y, int4 *dy, int V,
                                               int first, int step, int pr, float wj,
                                               unsigned &vmask, float &mine)
{
    const int lane = threadIdx.x & 31;
    int rows[ROWS];
    float w[ROWS], acc[ROWS];
    unsigned m = vmask;
#pragma unroll
    for (int b = 0; b < ROWS; b++, m &= m - 1) {
        const int j = m ? __ffs(m) - 1 : 0;
        const int row = __shfl_sync(kFull, pr, j);
        rows[b] = m ? row : -1;
        w[b] = __shfl_sync(kFull, wj, j);
        acc[b] = 0.f;
    }
    rows_backward<ROWS>(g, y, dy, V, first, step, rows, w, acc);
#pragma unroll
    for (int b = 0; b < ROWS; b++, vmask &= vmask - 1) {
        float a = acc[b];
#pragma unroll
        for (int off = 16; off; off >>= 1) a += __shfl_xor_sync(kFull, a, off);
        if (lane == __ffs(vmask) - 1) mine = a;
    }
}

// TEAM warps share a token: 1, or all of the CTA.
template <int TEAM, int ROWS>
__global__ void __launch_bounds__(kCbThreads, kCbCtas) k_combine_backward(
    const int4 *__restrict__ dout, const int4 *__restrict__ y, int y_rows,
    const int32_t *__restrict__ pair_row, const float *__restrict__ w,
    const int32_t *__restrict__ recv_pair, int64_t N, int k, int V, int4 *__restrict__ dy,
    float *__restrict__ dw, uint32_t *dev_status)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float part[TEAM > 1 ? TEAM : 1][32];
    bool bad_row = false;
    const int lane = threadIdx.x & 31, member = TEAM > 1 ? threadIdx.x >> 5 : 0;
    const int64_t gwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t gw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    // The CTA's tokens are n0 .. n1 - 1, one warp each (TEAM 1: the warp that is free next,
    // since tokens have different numbers of rows; a fixed share of them left the last
    // warps with twice the mean).  The next token's rows and weights are loaded while this
    // one's are worked on.
    __shared__ int taken;
    if (TEAM == 1 && threadIdx.x == 0) taken = kCbWarps;
    const unsigned base = (unsigned)N / gridDim.x, more = (unsigned)N - base * gridDim.x;   // N < 2^31
    const int64_t n0 = (int64_t)blockIdx.x * base + min(blockIdx.x, more);
    const int64_t n1 = n0 + base + (blockIdx.x < more);
    int64_t next = n0 + (TEAM == 1 ? threadIdx.x >> 5 : 0);
    auto take = [&]() {
        if (TEAM > 1) return next + 1;
        if (n1 - n0 <= kCbWarps) return n1;      // one each
        int t = 0;
        if (lane == 0) t = atomicAdd(&taken, 1);
        return n0 + __shfl_sync(kFull, t, 0);
    };
    int next_row = -1;
    float next_w = 0.f;
    auto load = [&](int64_t n) {
        next_row = -1;
        next_w = 0.f;
        if (n < n1 && lane < k) {
            next_row = __ldg(pair_row + n * k + lane);
            next_w = __ldg(w + n * k + lane);
        }
    };
    load(next);
    __syncthreads();
    while (next < n1) {
        const int64_t n = next;
        int pr = next_row;
        const float wj = next_w;
        next = take();
        load(next);
        if (pr >= y_rows) {
            bad_row = true;
            pr = -1;
        }
        unsigned vmask = __ballot_sync(kFull, pr >= 0);
        float mine = 0.f;             // lane j: gradient of weight j
        const int4 *g = dout + n * V;
        const int first = member * 32 + lane, step = TEAM * 32;
        while (vmask) {
            batch_backward<ROWS>(g, y, dy, V, first, step, pr, wj, vmask, mine);
        }
        if constexpr (TEAM > 1) {
            part[member][lane] = mine;
            __syncthreads();
            if (member == 0) {
                mine = 0.f;
#pragma unroll
                for (int m = 0; m < TEAM; m++) mine += part[m][lane];
            }
            __syncthreads();
        }
        if (member == 0 && lane < k) dw[n * k + lane] = mine;
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

template <int TEAM, int ROWS>
cudaError_t combine_backward(const uint16_t *d_out, const uint16_t *y, int y_rows,
                             const int32_t *pair_row, const float *w, const int32_t *recv_pair,
                             int64_t N, int k, int H, uint16_t *d_y, float *d_w,
                             uint32_t *dev_status, cudaStream_t st)
{
    const int64_t marks = recv_pair ? (y_rows + 31) / 32 : 0;
    const int64_t warps = N * TEAM > marks ? N * TEAM : marks;
    if (warps == 0) return cudaSuccess;
    const int64_t want = (warps + kCbWarps - 1) / kCbWarps;
    const int64_t fit = resident_grid((const void *)k_combine_backward<TEAM, ROWS>, kCbThreads, 0);
    const int64_t grid = fit > 0 && want > fit ? fit : want;
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_combine_backward", st,
        err = launch_pdl(k_combine_backward<TEAM, ROWS>, dim3((unsigned)grid), dim3(kCbThreads), 0, st,
                         (const int4 *)d_out, (const int4 *)y, y_rows, pair_row, w, recv_pair, N, k,
                         H / 8, (int4 *)d_y, d_w, dev_status));
    return err;
}

}  // namespace

cudaError_t launch_combine_backward(const uint16_t *d_out, const uint16_t *y, int y_rows,
                                    const int32_t *pair_row, const float *w,
                                    const int32_t *recv_pair, int64_t N, int k, int H,
                                    uint16_t *d_y, float *d_w, uint32_t *dev_status,
                                    cudaStream_t st)
{
    DeviceInfo di;
    const cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    // a CTA per token while its warps' columns hold a vector a lane and the tokens
    // alone do not fill the SMs
    const bool team = H >= 8 * kCbThreads && N <= 8 * di.sm_count;
    const bool many = k > 2 && y_rows > 2 * N;
#define CALL(TEAM, ROWS)                                                                       \
    combine_backward<TEAM, ROWS>(d_out, y, y_rows, pair_row, w, recv_pair, N, k, H, d_y, d_w,  \
                                 dev_status, st)
    if (team) return many ? CALL(kCbWarps, kManyRows) : CALL(kCbWarps, kFewRows);
    return many ? CALL(1, kManyRows) : CALL(1, kFewRows);
#undef CALL
}

}  // namespace moe
