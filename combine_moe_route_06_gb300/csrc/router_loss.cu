// router_loss.cu -- the router's training side: balance and z loss with
// per-expert counts, and the gradient of both and of the routing weights.
//
// For source s with valid tokens V (n = |V|), p_t = softmax(l_t), lse_t =
// log sum exp l_t:
//   c_e = picks of expert e by tokens of V,  P_e = (1/n) sum_{t in V} p_te
//   balance = (1/S) sum_s E/(k n) sum_e c_e P_e,  z = (1/S) sum_s (1/n) sum_t lse_t^2
// and, with d0, d1 the losses' gradients, A_e = d0 E/(k S n^2) c_e, g_j the
// gradient of routing weight j (softmax over the chosen logits):
//   dl_te = p_te (A_e - sum_i A_i p_ti + 2 d1 lse_t / (S n))
//           + [e = id_j] w_j (g_j - sum_i w_i g_i)
// The picks are constants of the gradient (a count has none).
//
// Logits are read once (and their gradient written once), so long batches are bound by
// memory and short ones by launches and one row's chain of reductions: 8 x 4,096 x 384
// padded logits take 18 us in the losses, 4,096 x 384 take 4.5 us in the gradient.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "trace.h"

namespace moe {

namespace {

constexpr int kRlThreads = 256;
constexpr int kRlWarps = kRlThreads / 32;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_as(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// exp(d) of a distance d <= 0 from the largest logit.  The error of the fast form
// grows with |d|, to 2^-22 |d| relative, where the probability is exp(d) small:
// below 2^-23 of the largest probability.
__device__ __forceinline__ float exp_below(float d) { return __expf(d); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int off = 16; off; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
    return v;
}

// Workspace of one call: per source and CTA the sums of the probabilities, the
// pick counts, the sum of lse^2 and the number of valid tokens; then what the
// second kernel's CTAs (one per source and 32 experts) hand to the last of them.
struct LossWs {
    float *prob;       // [S][B][E]
    int32_t *picks;    // [S][B][E]
    float *z;          // [S][B]
    int32_t *valid;    // [S][B]
    float *balance;    // [S][ceil(E / 32)]
    float *z_mean;     // [S]
    int32_t *arrived;  // [1]
};

// CTAs per source: two rows a warp where there are few, else about two CTAs per SM
// over all sources (four took 1.7 us more on 8 x 4,096 x 384 logits: more parts).
int loss_ctas(int S, int T)
{
    const int by_rows = (T + 15) / 16;
    const int by_grid = S >= 304 ? 1 : 304 / S;
    const int b = by_rows < by_grid ? by_rows : by_grid;
    return b < 1 ? 1 : b;
}
int loss_blocks(int E) { return (E + 31) / 32; }

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

LossWs carve(void *ws, int S, int B, int E)
{
    char *p = (char *)ws;
    LossWs w;
    w.prob = (float *)p;
    p += align256((size_t)S * B * E * 4);
    w.picks = (int32_t *)p;
    p += align256((size_t)S * B * E * 4);
    w.z = (float *)p;
    p += align256((size_t)S * B * 4);
    w.valid = (int32_t *)p;
    p += align256((size_t)S * B * 4);
    w.balance = (float *)p;
    p += align256((size_t)S * loss_blocks(E) * 4);
    w.z_mean = (float *)p;
    p += align256((size_t)S * 4);
    w.arrived = (int32_t *)p;
    return w;
}

// A call of one source and at most kOneRows tokens is one launch of one cluster,
// whose CTAs' sums are joined in distributed shared memory; else the CTAs' sums go
// through the workspace to a second kernel (128 x 16 logits: 3.9 us in one launch,
// 6.1 in two; 256 x 384: 6.1 and 7.4; 512 x 384: 8.6 and 7.4).
constexpr int kOneCtas = 8;
constexpr int kOneRows = 256;

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
template <typename T>
__device__ __forceinline__ const T *of_cta(const T *p, int rank)
{
    return (const T *)__cluster_map_shared_rank(p, rank);
}

// Warps per CTA of the first kernel: 16 where a row takes few registers (8 x 4,096 x
// 384 logits: 19.5 us, 20.4 with 8).
constexpr int part_warps(int vpl) { return vpl <= 12 ? 16 : 8; }

struct LossOut {
    int32_t *counts;
    float *prob_mean;
    int32_t *n_valid;
    float *losses;
};

// One warp per token: the row in registers, its softmax added to the lane's
// column sums; the CTA's sums go to the workspace, or with ONE to the cluster's
// first CTA, which writes the results.
template <typename L, int VPL, bool ONE>
__global__ void __launch_bounds__(part_warps(VPL) * 32, 2) k_balance_part(
    const L *__restrict__ logits, const int32_t *__restrict__ ids,
    const uint8_t *__restrict__ mask, int T, int E, int k, float *__restrict__ lse, LossWs ws,
    LossOut out, uint32_t *dev_status)
{
    constexpr int W = part_warps(VPL);
    pdl_wait();
    pdl_trigger();
    extern __shared__ float sm[];              // [warps][E] sums, then [E] picks
    int32_t *picks = (int32_t *)(sm + W * E);
    __shared__ float zsum[W];
    __shared__ int nsum[W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = blockIdx.y, b = blockIdx.x, B = gridDim.x;
    for (int e = threadIdx.x; e < E; e += (W * 32)) picks[e] = 0;
    if (!ONE && s == 0 && b == 0 && threadIdx.x == 0) *ws.arrived = 0;
    __syncthreads();

    float acc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i++) acc[i] = 0.f;
    float z = 0.f;
    int n = 0;
    bool bad_id = false;
    // the next row's loads are in flight while this one is summed, and the mark of
    // the row after it, so that rows that are not valid are never loaded
    struct Row {
        L v[VPL];
        int id;
        bool valid;
    } next;
    const int64_t step = B * W;
    auto valid = [&](int64_t t) { return t < T && (mask == nullptr || mask[(int64_t)s * T + t] != 0); };
    auto load = [&](int64_t t, bool marked, Row &r) {
        r.valid = marked;
        r.id = -1;
        if (!marked) return;
        const int64_t row = (int64_t)s * T + t;
        if (lane < k) r.id = __ldg(ids + row * k + lane);
        const L *src = logits + row * E;
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (lane + 32 * i < E) r.v[i] = src[lane + 32 * i];
    };
    const int64_t t0 = b * W + warp;
    load(t0, valid(t0), next);
    bool marked = valid(t0 + step);
    for (int64_t t = t0; t < T; t += step) {
        const Row now = next;
        load(t + step, marked, next);
        marked = valid(t + 2 * step);
        const int64_t row = (int64_t)s * T + t;
        if (!now.valid) {
            if (lane == 0) lse[row] = 0.f;
            continue;
        }
        n++;
        if (now.id >= E) bad_id = true;
        else if (now.id >= 0) atomicAdd(&picks[now.id], 1);
        float v[VPL];
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            v[i] = lane + 32 * i < E ? to_float(now.v[i]) : -INFINITY;
            top = fmaxf(top, v[i]);
        }
        top = warp_max(top);
        const float base = top == -INFINITY ? 0.f : top;   // a row of -inf: all terms 0
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            v[i] = exp_below(v[i] - base);
            sum += v[i];
        }
        sum = warp_sum(sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < VPL; i++) acc[i] = fmaf(v[i], inv, acc[i]);
        const float l = base + logf(sum);
        if (sum != 0.f) z = fmaf(l, l, z);
        if (lane == 0) lse[row] = l;
    }
    if (bad_id) flag_status(dev_status, MOE_ERR_BAD_EXPERT_ID);
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        if (e < E) sm[warp * E + e] = acc[i];
    }
    if (lane == 0) {
        zsum[warp] = z;
        nsum[warp] = n;
    }
    __syncthreads();
    const int64_t at = (int64_t)s * B + b;
    for (int e = threadIdx.x; e < E; e += (W * 32)) {
        float p = 0.f;
#pragma unroll
        for (int w = 0; w < W; w++) p += sm[w * E + e];
        if constexpr (ONE) {
            sm[e] = p;
        } else {
            ws.prob[at * E + e] = p;
            ws.picks[at * E + e] = picks[e];
        }
    }
    if (threadIdx.x == 0) {
        float zt = 0.f;
        int nt = 0;
        for (int w = 0; w < W; w++) {
            zt += zsum[w];
            nt += nsum[w];
        }
        if constexpr (ONE) {
            zsum[0] = zt;
            nsum[0] = nt;
        } else {
            ws.z[at] = zt;
            ws.valid[at] = nt;
        }
    }
    if constexpr (ONE) {
        cluster_barrier();
        if (b == 0) {
            int nt = 0;
            float zt = 0.f;
#pragma unroll
            for (int r = 0; r < kOneCtas; r++) {
                nt += *of_cta(nsum, r);
                zt += *of_cta(zsum, r);
            }
            const float inv = nt > 0 ? 1.f / (float)nt : 0.f;
            float dot = 0.f;
            for (int e = threadIdx.x; e < E; e += (W * 32)) {
                float p = 0.f;
                int c = 0;
#pragma unroll
                for (int r = 0; r < kOneCtas; r++) {
                    p += *of_cta(sm + e, r);
                    c += *of_cta(picks + e, r);
                }
                p *= inv;
                out.counts[e] = c;
                out.prob_mean[e] = p;
                dot = fmaf((float)c, p, dot);
            }
            dot = warp_sum(dot);
            __shared__ float dots[W];
            if (lane == 0) dots[warp] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                float d = 0.f;
                for (int w = 0; w < W; w++) d += dots[w];
                *out.n_valid = nt;
                out.losses[0] = d * inv * ((float)E / (float)k);
                out.losses[1] = zt * inv;
            }
        }
        cluster_barrier();      // the other CTAs' shared memory stays until it has been read
    }
}

// One CTA per source and 32 experts sums the parts in their order; the last CTA
// to arrive adds the losses up, in order again.
__global__ void __launch_bounds__(kRlThreads) k_balance_finish(LossWs ws, int S, int B, int E, int k,
                                                               int32_t *__restrict__ counts,
                                                               float *__restrict__ prob_mean,
                                                               int32_t *__restrict__ n_valid,
                                                               float *__restrict__ losses)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float prob[kRlWarps][32];
    __shared__ int picks[kRlWarps][32];
    __shared__ int n_sh;
    __shared__ float z_sh;
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int block = blockIdx.x, blocks = gridDim.x, s = blockIdx.y;
    const int e = block * 32 + lane;
    float p = 0.f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
        for (int b = warp; b < B; b += kRlWarps) {
            p += ws.prob[((int64_t)s * B + b) * E + e];
            c += ws.picks[((int64_t)s * B + b) * E + e];
        }
    }
    prob[warp][lane] = p;
    picks[warp][lane] = c;
    if (warp == 1) {
        int n = 0;
        for (int b = lane; b < B; b += 32) n += ws.valid[(int64_t)s * B + b];
        n = __reduce_add_sync(kFull, n);
        if (lane == 0) n_sh = n;
    } else if (warp == 2) {
        float z = 0.f;
        for (int b = lane; b < B; b += 32) z += ws.z[(int64_t)s * B + b];
        z = warp_sum(z);
        if (lane == 0) z_sh = z;
    }
    __syncthreads();
    if (warp != 0) return;
    const int n = n_sh;
    const float inv = n > 0 ? 1.f / (float)n : 0.f;
    p = 0.f;
    c = 0;
#pragma unroll
    for (int w = 0; w < kRlWarps; w++) {
        p += prob[w][lane];
        c += picks[w][lane];
    }
    p *= inv;
    if (e < E) {
        counts[(int64_t)s * E + e] = c;
        prob_mean[(int64_t)s * E + e] = p;
    }
    const float dot = warp_sum((float)c * p);
    if (lane == 0) {
        ws.balance[(int64_t)s * blocks + block] = dot * inv * ((float)E / (float)k);
        if (block == 0) {
            n_valid[s] = n;
            ws.z_mean[s] = z_sh * inv;
        }
        __threadfence();
        last = atomicAdd(ws.arrived, 1) == blocks * S - 1;
    }
    __syncwarp();
    if (!last) return;
    __threadfence();
    float balance = 0.f, z = 0.f;
    for (int i = lane; i < S * blocks; i += 32) balance += __ldcg(ws.balance + i);
    for (int i = lane; i < S; i += 32) z += __ldcg(ws.z_mean + i);
    balance = warp_sum(balance);
    z = warp_sum(z);
    if (lane == 0) {
        losses[0] = balance / (float)S;
        losses[1] = z / (float)S;
    }
}

// One warp per token.  With LOSS the dense part is computed from the logits and
// the saved lse, else it is zero; the chosen experts' entries are then stored
// once more with the routing weights' part added (a warp barrier orders the
// two stores of an element).
template <typename L, int VPL, bool LOSS>
__global__ void __launch_bounds__(kRlThreads) k_route_backward(
    const L *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ w,
    const float *__restrict__ dw, const float *__restrict__ lse, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ n_valid, const float *__restrict__ d_losses,
    const uint8_t *__restrict__ mask, int S, int T, int E, int k, L *__restrict__ out,
    uint32_t *dev_status)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t N = (int64_t)S * T;
    const int64_t stride = (int64_t)gridDim.x * kRlWarps;
    bool bad_id = false;
    for (int64_t row = (int64_t)blockIdx.x * kRlWarps + (threadIdx.x >> 5); row < N;
         row += stride) {
        L *dst = out + row * E;
        if (mask && mask[row] == 0) {
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int e = lane + 32 * i;
                if (e < E) store_as(dst + e, 0.f);
            }
            continue;
        }
        const int s = (int)(row / T);
        int id = -1;
        float g = 0.f;
        if (w) {
            float wj = 0.f, gj = 0.f;
            if (lane < k) {
                id = __ldg(ids + row * k + lane);
                wj = __ldg(w + row * k + lane);
                gj = __ldg(dw + row * k + lane);
                if (id >= E) bad_id = true;
                if (id < 0 || id >= E) {
                    id = -1;
                    wj = 0.f;
                    gj = 0.f;
                }
            }
            const float dot = warp_sum(wj * gj);
            g = wj * (gj - dot);
        }
        if constexpr (LOSS) {
            const float n = fmaxf((float)__ldg(n_valid + s), 1.f);
            const float per = 1.f / ((float)S * n);
            const float lead = __ldg(d_losses) * ((float)E / (float)k) * per / n;
            const float l = __ldg(lse + row);
            const bool empty = l == -INFINITY;     // a row of -inf has no gradient
            const float zc = empty ? 0.f : 2.f * __ldg(d_losses + 1) * per * l;
            const L *src = logits + row * E;
            const int32_t *c = counts + (int64_t)s * E;
            // the softmax again from the row: exp(l - lse) would carry the rounding of lse
            float p[VPL], a[VPL];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int e = lane + 32 * i;
                p[i] = e < E ? to_float(src[e]) : -INFINITY;
                a[i] = e < E ? lead * (float)__ldg(c + e) : 0.f;
                top = fmaxf(top, p[i]);
            }
            top = warp_max(top);
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                p[i] = exp_below(p[i] - base);
                sum += p[i];
            }
            sum = warp_sum(sum);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                p[i] *= inv;
                dot = fmaf(a[i], p[i], dot);
            }
            const float back = zc - warp_sum(dot);
            float chosen = 0.f;
            if (id >= 0) {
                const float q = exp_below(to_float(src[id]) - base) * inv;
                chosen = q * (lead * (float)__ldg(c + id) + back);
            }
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int e = lane + 32 * i;
                if (e < E) store_as(dst + e, p[i] * (a[i] + back));
            }
            if (w) {
                for (int j = 0; j < k; j++) {      // picks of the same expert add up
                    const int ij = __shfl_sync(kFull, id, j);
                    const float gj = __shfl_sync(kFull, g, j);
                    if (ij == id) chosen += gj;
                }
                __syncwarp();
                if (id >= 0) store_as(dst + id, chosen);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int e = lane + 32 * i;
                if (e < E) store_as(dst + e, 0.f);
            }
            if (w) {
                float chosen = 0.f;
                for (int j = 0; j < k; j++) {
                    const int ij = __shfl_sync(kFull, id, j);
                    const float gj = __shfl_sync(kFull, g, j);
                    if (ij == id) chosen += gj;
                }
                __syncwarp();
                if (id >= 0) store_as(dst + id, chosen);
            }
        }
    }
    if (bad_id) flag_status(dev_status, MOE_ERR_BAD_EXPERT_ID);
}

// The same for few experts (E <= 128, E a multiple of 4, k <= 8): eight lanes per
// token, each with NC vectors of four logits, so that a warp's reductions serve four
// tokens (16,384 x 64 in bf16: 4.6 us, 6.8 with a warp per token).
constexpr int kFewLanes = 8;

__device__ __forceinline__ void load_four(const float *p, float (&v)[4])
{
    const float4 q = *(const float4 *)p;
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
}
__device__ __forceinline__ void load_four(const __nv_bfloat16 *p, float (&v)[4])
{
    const uint2 q = *(const uint2 *)p;
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void store_four(float *p, const float (&v)[4])
{
    *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_four(__nv_bfloat16 *p, const float (&v)[4])
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *(uint2 *)p = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ float eight_sum(float v)
{
#pragma unroll
    for (int off = kFewLanes / 2; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

template <typename L, int NC, bool LOSS>
__global__ void __launch_bounds__(kRlThreads) k_route_backward_few(
    const L *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ w,
    const float *__restrict__ dw, const float *__restrict__ lse, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ n_valid, const float *__restrict__ d_losses,
    const uint8_t *__restrict__ mask, int S, int T, int E, int k, L *__restrict__ out,
    uint32_t *dev_status)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kTokens = 32 / kFewLanes;
    const int lane = threadIdx.x & 31, sub = lane % kFewLanes;
    const int64_t N = (int64_t)S * T;
    const int64_t stride = (int64_t)gridDim.x * kRlWarps * kTokens;
    bool bad_id = false;
    float d0 = 0.f, d1 = 0.f;
    if (LOSS) {
        d0 = __ldg(d_losses) * ((float)E / (float)k);
        d1 = 2.f * __ldg(d_losses + 1);
    }
    for (int64_t row0 = ((int64_t)blockIdx.x * kRlWarps + (threadIdx.x >> 5)) * kTokens; row0 < N;
         row0 += stride) {
        const int64_t row = row0 + lane / kFewLanes;
        const bool live = row < N, valid = live && (mask == nullptr || mask[row] != 0);
        const int s = live ? (int)(row / T) : 0;
        int id = -1;
        float wj = 0.f, gj = 0.f, l = 0.f, n = 1.f;
        float p[NC][4], a[NC][4];
        if (w && valid && sub < k) {
            id = __ldg(ids + row * k + sub);
            wj = __ldg(w + row * k + sub);
            gj = __ldg(dw + row * k + sub);
            if (id >= E) bad_id = true;
            if (id < 0 || id >= E) {
                id = -1;
                wj = 0.f;
                gj = 0.f;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int e = 4 * (sub + kFewLanes * c);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                p[c][i] = -INFINITY;
                a[c][i] = 0.f;
            }
            if (LOSS && valid && e < E) {
                load_four(logits + row * E + e, p[c]);
                const int4 q = __ldg((const int4 *)(counts + (int64_t)s * E + e));
                a[c][0] = (float)q.x, a[c][1] = (float)q.y, a[c][2] = (float)q.z, a[c][3] = (float)q.w;
            }
#pragma unroll
            for (int i = 0; i < 4; i++) top = fmaxf(top, p[c][i]);
        }
        if (LOSS && valid) {
            l = __ldg(lse + row);
            n = fmaxf((float)__ldg(n_valid + s), 1.f);
        }
        const float g = wj * (gj - eight_sum(wj * gj));
        float chosen = 0.f;                      // picks of the same expert add up
        for (int j = 0; j < k && w; j++) {
            const int ij = __shfl_sync(kFull, id, j, kFewLanes);
            const float other = __shfl_sync(kFull, g, j, kFewLanes);
            if (ij == id) chosen += other;
        }
        float back = 0.f, inv = 0.f, lead = 0.f, base = 0.f;
        if constexpr (LOSS) {
            const float per = 1.f / ((float)S * n);
            lead = d0 * per / n;
            // the softmax again from the row: exp(l - lse) would carry the rounding of lse
#pragma unroll
            for (int off = kFewLanes / 2; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
            base = top == -INFINITY ? 0.f : top;
            float sum = 0.f, dot = 0.f;
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    p[c][i] = exp_below(p[c][i] - base);
                    sum += p[c][i];
                    a[c][i] *= lead;
                }
            sum = eight_sum(sum);
            inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    p[c][i] *= inv;
                    dot = fmaf(a[c][i], p[c][i], dot);
                }
            // (a row of -inf has no gradient)
            back = (l == -INFINITY ? 0.f : d1 * per * l) - eight_sum(dot);
            if (id >= 0) {
                const float q = exp_below(to_float(logits[row * E + id]) - base) * inv;
                chosen += q * (lead * (float)__ldg(counts + (int64_t)s * E + id) + back);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int e = 4 * (sub + kFewLanes * c);
            float r[4];
#pragma unroll
            for (int i = 0; i < 4; i++) r[i] = LOSS && valid ? p[c][i] * (a[c][i] + back) : 0.f;
            if (live && e < E) store_four(out + row * E + e, r);
        }
        __syncwarp();
        if (id >= 0) store_as(out + row * E + id, chosen);
    }
    if (bad_id) flag_status(dev_status, MOE_ERR_BAD_EXPERT_ID);
}

// VPL: logits per lane, the smallest instance that holds E.
#define MOE_VPL_CASES(E, CALL)          \
    do {                                \
        const int vpl_ = ((E) + 31) / 32; \
        if (vpl_ <= 1) { CALL(1); }     \
        else if (vpl_ <= 2) { CALL(2); } \
        else if (vpl_ <= 4) { CALL(4); } \
        else if (vpl_ <= 8) { CALL(8); } \
        else if (vpl_ <= 12) { CALL(12); } \
        else if (vpl_ <= 16) { CALL(16); } \
        else if (vpl_ <= 24) { CALL(24); } \
        else { CALL(32); }              \
    } while (0)

template <typename L>
cudaError_t balance_part(const L *logits, const int32_t *ids, const uint8_t *mask, int S, int T,
                         int E, int k, int B, bool one, float *lse, LossWs ws, LossOut out,
                         uint32_t *dev_status, cudaStream_t st)
{
    auto smem = [&](int v) { return (size_t)(part_warps(v) + 1) * E * 4; };
    cudaError_t err = cudaSuccess;
#define CALL(V)                                                                                    \
    if (one)                                                                                       \
        MOE_TRACED_LAUNCH("k_balance_part", st,                                                    \
            err = launch_pdl_cluster(k_balance_part<L, V, true>, dim3(kOneCtas), dim3(part_warps(V) * 32), \
                                     smem(V), kOneCtas, st, logits, ids, mask, T, E, k, lse, ws, out,  \
                                     dev_status));                                                 \
    else                                                                                           \
        MOE_TRACED_LAUNCH("k_balance_part", st,                                                    \
            err = launch_pdl(k_balance_part<L, V, false>, dim3(B, S), dim3(part_warps(V) * 32), smem(V), st,  \
                             logits, ids, mask, T, E, k, lse, ws, out, dev_status))
    MOE_VPL_CASES(E, CALL);
#undef CALL
    return err;
}

template <typename L>
cudaError_t route_backward(const L *logits, const int32_t *ids, const float *w, const float *dw,
                           const float *lse, const int32_t *counts, const int32_t *n_valid,
                           const float *d_losses, const uint8_t *mask, int S, int T, int E, int k,
                           L *out, uint32_t *dev_status, cudaStream_t st)
{
    const int64_t N = (int64_t)S * T;
    auto vectors = [](const void *p, size_t size) { return (uintptr_t)p % (4 * size) == 0; };
    if (E <= 128 && E % 4 == 0 && k <= kFewLanes && vectors(out, sizeof(L)) &&
        (!d_losses || (vectors(logits, sizeof(L)) && vectors(counts, 4)))) {
        const int64_t want = (N + kRlWarps * 4 - 1) / (kRlWarps * 4);
        cudaError_t err;
#define CALL2(NC, LOSS)                                                                           \
    do {                                                                                          \
        const int64_t fit =                                                                       \
            resident_grid((const void *)k_route_backward_few<L, NC, LOSS>, kRlThreads, 0);        \
        const int64_t grid = fit > 0 && want > fit ? fit : want;                                  \
        MOE_TRACED_LAUNCH("k_route_backward", st,                                                 \
            err = launch_pdl(k_route_backward_few<L, NC, LOSS>, dim3((unsigned)grid),             \
                             dim3(kRlThreads), 0, st, logits, ids, w, dw, lse, counts, n_valid,   \
                             d_losses, mask, S, T, E, k, out, dev_status));                       \
    } while (0)
#define CALL(NC) if (d_losses) CALL2(NC, true); else CALL2(NC, false)
        if (E <= 32) { CALL(1); }
        else if (E <= 64) { CALL(2); }
        else { CALL(4); }
#undef CALL
#undef CALL2
        return err;
    }
    const int64_t want = (N + kRlWarps - 1) / kRlWarps;
    cudaError_t err = cudaSuccess;
#define CALL2(V, LOSS)                                                                          \
    do {                                                                                        \
        const int64_t fit = resident_grid((const void *)k_route_backward<L, V, LOSS>, kRlThreads, 0); \
        const int64_t grid = fit > 0 && want > fit ? fit : want;                                \
        MOE_TRACED_LAUNCH("k_route_backward", st,                                               \
            err = launch_pdl(k_route_backward<L, V, LOSS>, dim3((unsigned)grid), dim3(kRlThreads), \
                             0, st, logits, ids, w, dw, lse, counts, n_valid, d_losses, mask, S, T, \
                             E, k, out, dev_status));                                           \
    } while (0)
#define CALL(V) if (d_losses) CALL2(V, true); else CALL2(V, false)
    MOE_VPL_CASES(E, CALL);
#undef CALL
#undef CALL2
    return err;
}

}  // namespace

size_t balance_loss_ws_bytes(int S, int T, int E)
{
    const int B = loss_ctas(S, T);
    return 2 * align256((size_t)S * B * E * 4) + 2 * align256((size_t)S * B * 4) +
           align256((size_t)S * loss_blocks(E) * 4) + align256((size_t)S * 4) + 256;
}

cudaError_t launch_balance_loss(const void *logits, int type, const int32_t *ids,
                                const uint8_t *mask, int S, int T, int E, int k, int32_t *counts,
                                float *prob_mean, float *lse, int32_t *n_valid, float *losses,
                                void *ws, uint32_t *dev_status, cudaStream_t st)
{
    const int B = loss_ctas(S, T);
    const bool one = S == 1 && T <= kOneRows;
    const LossWs w = carve(ws, S, B, E);
    const LossOut out{counts, prob_mean, n_valid, losses};
    cudaError_t err = type == MOE_TYPE_BF16
                          ? balance_part((const __nv_bfloat16 *)logits, ids, mask, S, T, E, k, B, one,
                                         lse, w, out, dev_status, st)
                          : balance_part((const float *)logits, ids, mask, S, T, E, k, B, one, lse, w,
                                         out, dev_status, st);
    if (err != cudaSuccess || one) return err;
    MOE_TRACED_LAUNCH("k_balance_finish", st,
        err = launch_pdl(k_balance_finish, dim3(loss_blocks(E), S), dim3(kRlThreads), 0, st, w, S, B,
                         E, k, counts, prob_mean, n_valid, losses));
    return err;
}

cudaError_t launch_route_backward(const void *logits, int type, const int32_t *ids, const float *w,
                                  const float *dw, const float *lse, const int32_t *counts,
                                  const int32_t *n_valid, const float *d_losses,
                                  const uint8_t *mask, int S, int T, int E, int k, void *d_logits,
                                  uint32_t *dev_status, cudaStream_t st)
{
    if ((int64_t)S * T == 0) return cudaSuccess;
    if (type == MOE_TYPE_BF16)
        return route_backward((const __nv_bfloat16 *)logits, ids, w, dw, lse, counts, n_valid,
                              d_losses, mask, S, T, E, k, (__nv_bfloat16 *)d_logits, dev_status, st);
    return route_backward((const float *)logits, ids, w, dw, lse, counts, n_valid, d_losses, mask,
                          S, T, E, k, (float *)d_logits, dev_status, st);
}

}  // namespace moe
