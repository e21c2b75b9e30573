// expert_product.cu -- the experts' products with bf16 weights and their gradients.
//
// Three products over the rows of each expert e (W_e [N][K]):
//   y[r][n]   = sum_k a[r][k] W_e[n][k]      (gated: silu of one sum times another)
//   d_a[r][k] = sum_n d_y[r][n] W_e[n][k]    (or the gradient in gate and up)
//   d_w[n][k] = sum_r d_y[r][n] a[r][k]
// each a sum over l of X(i, l) Y(j, l): one kernel of 64 x 64 outputs a CTA in turn, both
// operands staged in shared memory, sums in fp32 registers.
#include <cuda_bf16.h>

#include "common.cuh"
#include "gate.cuh"
#include "launch.h"
#include "trace.h"
#include "w4.cuh"

namespace moe {

namespace {

constexpr int kTile = 64, kStep = 16, kMmThreads = 256;

enum Form { kPlain, kGated, kRowGrad, kGateGrad, kWeightGrad };

struct Args {
    const __nv_bfloat16 *x, *y;     // the operands: i is a row or an output, j likewise
    const int32_t *offsets, *counts;
    int block_rows, a_rows, E, N, K;
    __nv_bfloat16 *out;
    const __nv_bfloat16 *pre;       // in (gradient in gate and up)
    __nv_bfloat16 *keep;            // out (gated)
    void *d_w;
    bool d_w_f32;
    uint32_t *dev_status;
};

template <int FORM>
__global__ void __launch_bounds__(kMmThreads) k_expert_product(const __grid_constant__ Args p)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float xs[kStep][kTile + 1], ys[FORM == kGated ? 2 : 1][kStep][kTile + 1];
    const int e = blockIdx.y, tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    int start, count;
    bool bad = false;
    expert_rows(p.offsets, p.counts, p.block_rows, p.a_rows, e, start, count, bad);
    if (p.offsets && p.offsets[e + 1] < p.offsets[e]) bad = true;
    if (bad && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) flag_status(p.dev_status, MOE_ERR_INVALID_ARG);
    // outputs I x J, sums over L; element (i, l) of x at xi * i + xl * l, of y likewise
    const bool grad = FORM == kRowGrad || FORM == kGateGrad, weights = FORM == kWeightGrad;
    const int I = weights ? p.N : count, J = weights || grad ? p.K : p.N;
    const int L = weights ? count : grad ? p.N : p.K;
    const int64_t xi = weights ? 1 : grad ? p.N : p.K, xl = weights ? p.N : 1;
    const int64_t yj = weights || grad ? 1 : p.K, yl = weights || grad ? p.K : 1;
    const __nv_bfloat16 *x = p.x + (int64_t)start * (weights || grad ? p.N : p.K);
    const __nv_bfloat16 *y = p.y + (weights ? (int64_t)start * p.K
                                            : (int64_t)e * (FORM == kGated ? 2 : 1) * p.N * p.K);
    const int j0 = blockIdx.x * kTile;
    for (int i0 = blockIdx.z * kTile; i0 < I; i0 += gridDim.z * kTile) {
        float acc[FORM == kGated ? 2 : 1][4][4] = {};
        for (int l0 = 0; l0 < L; l0 += kStep) {
            for (int at = tid; at < kTile * kStep; at += kMmThreads) {
                const int l = weights ? at / kTile : at % kStep, i = weights ? at % kTile : at / kStep;
                xs[l][i] = i0 + i < I && l0 + l < L ? __bfloat162float(x[(i0 + i) * xi + (l0 + l) * xl]) : 0.f;
            }
            for (int at = tid; at < kTile * kStep; at += kMmThreads) {
                const int l = yj == 1 ? at / kTile : at % kStep, j = yj == 1 ? at % kTile : at / kStep;
                for (int h = 0; h < (FORM == kGated ? 2 : 1); h++)
                    ys[h][l][j] = j0 + j < J && l0 + l < L
                                      ? __bfloat162float(y[((int64_t)h * p.N + j0 + j) * yj + (l0 + l) * yl])
                                      : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int l = 0; l < kStep; l++)
#pragma unroll
                for (int u = 0; u < 4; u++)
#pragma unroll
                    for (int v = 0; v < 4; v++)
#pragma unroll
                        for (int h = 0; h < (FORM == kGated ? 2 : 1); h++)
                            acc[h][u][v] = fmaf(xs[l][ty + 16 * u], ys[h][l][tx + 16 * v], acc[h][u][v]);
            __syncthreads();
        }
        for (int u = 0; u < 4; u++)
            for (int v = 0; v < 4; v++) {
                const int i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
                if (i >= I || j >= J) continue;
                const float s = acc[0][u][v];
                const int64_t r = start + i;
                if constexpr (FORM == kGated) {
                    const float up = acc[1][u][v];
                    p.out[r * J + j] = __float2bfloat16_rn(gated_output(s, up));
                    if (p.keep) {
                        p.keep[r * 2 * J + j] = __float2bfloat16_rn(s);
                        p.keep[r * 2 * J + J + j] = __float2bfloat16_rn(up);
                    }
                } else if constexpr (FORM == kGateGrad) {
                    const float g = __bfloat162float(p.pre[r * 2 * J + j]);
                    const float up = __bfloat162float(p.pre[r * 2 * J + J + j]);
                    float d_gate, d_up;
                    gated_gradient(g, up, s, d_gate, d_up);
                    p.out[r * 2 * J + j] = __float2bfloat16_rn(d_gate);
                    p.out[r * 2 * J + J + j] = __float2bfloat16_rn(d_up);
                } else if constexpr (FORM == kWeightGrad) {
                    const int64_t at = ((int64_t)e * I + i) * J + j;
                    if (p.d_w_f32) ((float *)p.d_w)[at] = s;
                    else ((__nv_bfloat16 *)p.d_w)[at] = __float2bfloat16_rn(s);
                } else {
                    p.out[r * J + j] = __float2bfloat16_rn(s);
                }
            }
    }
}

template <int FORM>
cudaError_t product(const Args &p, int J, int I, cudaStream_t st)
{
    const int deep = (I + kTile - 1) / kTile;
    const dim3 grid((J + kTile - 1) / kTile, p.E, deep < 1 ? 1 : deep < 64 ? deep : 64);
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_expert_product", st,
        err = launch_pdl(k_expert_product<FORM>, grid, dim3(kMmThreads), 0, st, p));
    return err;
}

}  // namespace

size_t expert_product_ws_bytes() { return 256; }

cudaError_t launch_expert_product(const uint16_t *a, int a_rows, const int32_t *offsets,
                                  const int32_t *counts, int block_rows, const uint16_t *w, int E,
                                  int N, int K, bool gated, uint16_t *y, uint16_t *pre, void *ws,
                                  uint32_t *dev_status, cudaStream_t st)
{
    (void)ws;
    if (a_rows == 0) return cudaSuccess;
    const Args p{(const __nv_bfloat16 *)a, (const __nv_bfloat16 *)w, offsets, counts, block_rows,
                 a_rows, E, N, K, (__nv_bfloat16 *)y, nullptr, (__nv_bfloat16 *)pre, nullptr, false,
                 dev_status};
    return gated ? product<kGated>(p, N, a_rows, st) : product<kPlain>(p, N, a_rows, st);
}

cudaError_t launch_expert_product_backward(const uint16_t *d_y, const uint16_t *a, int a_rows,
                                           const int32_t *offsets, const int32_t *counts,
                                           int block_rows, const uint16_t *w, const uint16_t *pre,
                                           int E, int N, int K, uint16_t *d_a, void *d_w,
                                           int d_w_type, void *ws, uint32_t *dev_status,
                                           cudaStream_t st)
{
    (void)ws;
    Args p{(const __nv_bfloat16 *)d_y, (const __nv_bfloat16 *)w, offsets, counts, block_rows,
           a_rows, E, N, K, (__nv_bfloat16 *)d_a, (const __nv_bfloat16 *)pre, nullptr, d_w,
           d_w_type == MOE_TYPE_F32, dev_status};
    cudaError_t err = cudaSuccess;
    if (d_a && a_rows > 0) err = pre ? product<kGateGrad>(p, K, a_rows, st) : product<kRowGrad>(p, K, a_rows, st);
    if (err != cudaSuccess || !d_w) return err;
    p.y = (const __nv_bfloat16 *)a;
    return product<kWeightGrad>(p, K, N, st);
}

}  // namespace moe
