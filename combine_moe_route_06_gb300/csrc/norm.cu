// norm.cu -- RMS norm with the residual's addition, rows out in bf16 and as MXFP8
// records, and its gradient.
//
//   h = x + residual,   inv = 1 / sqrt(mean(h^2) + eps),   y = h inv w
//
// Forward: a row is held in registers between the sum of squares and the output, so
// every input is read once and every output written once.  A team of warps has one row, and the
// next CTA the next ones (16,384 rows of 2,048 with an fp32 residual: 59.5 us, 6.8 TB/s; 69.7 by
// CTAs that stay and go on to further rows, whose loads then wait for the row before).  The
// record is the MXFP8 form of the row in bf16 (quant.cuh), the bytes that the quantized pack
// makes of y (4,096 rows of 5,120 with both outputs: 31 us, 6.1 TB/s).
//
// Backward, with q = d_y w:
//   d_h = d_residual + inv (q - h inv^2 mean(q h)),   d_w = sum over rows of d_y h inv
// sum(h^2) and sum(q h) come out of one pass over the row in registers.  A CTA adds its
// rows' parts of d_w in registers, writes them to the workspace, and a second kernel
// sums the CTAs' parts in their order.
//
// (16,384 rows of 5,120 with a residual's gradient: 104.7 us, 6.4 TB/s; rows wider than 8,192 are far from that,
// 1,500 of 30,000 208 us, 1.7 TB/s: no row is copied ahead, and 32 warps leave a thread too few registers.)
//
// Both are bound by HBM, but for those.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "quant.cuh"
#include "trace.h"

namespace moe {

namespace {

constexpr int kRowsWarps = 8;           // warps of a CTA that several teams share
constexpr int kMaxParts = 640;          // CTAs of the backward pass, and parts of d_w

// A row is shared by a team of WARPS warps, each thread with NV vectors of 8 values:
// vector i of thread t is columns 8 (t + i * 32 WARPS) on.  Small teams share a CTA.
template <int WARPS>
constexpr int kTeams = WARPS < kRowsWarps ? kRowsWarps / WARPS : 1;
template <int WARPS>
constexpr int kThreads = 32 * WARPS * kTeams<WARPS>;

__device__ __forceinline__ void unpack8(int4 v, float (&f)[8])
{
    const uint32_t u[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ int4 pack8(const float (&f)[8])
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_int4((int)r[0], (int)r[1], (int)r[2], (int)r[3]);
}

// Eight values at vector `v` of an array of fp32 or bf16, as loaded: two 16-byte words
// or one.
template <bool F32>
struct Raw8 {
    int4 w[F32 ? 2 : 1];
    __device__ void load(const void *p, int64_t v)
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); i++) w[i] = ld_stream((const int4 *)p + v * (F32 ? 2 : 1) + i);
    }
    __device__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); i++) w[i] = make_int4(0, 0, 0, 0);
    }
    __device__ void values(float (&f)[8]) const
    {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                f[4 * i] = __int_as_float(w[i].x);
                f[4 * i + 1] = __int_as_float(w[i].y);
                f[4 * i + 2] = __int_as_float(w[i].z);
                f[4 * i + 3] = __int_as_float(w[i].w);
            }
        } else {
            unpack8(w[0], f);
        }
    }
};
template <bool F32>
__device__ __forceinline__ void store8(void *p, int64_t v, const float (&f)[8])
{
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            st_stream((int4 *)p + 2 * v + i,
                      make_int4(__float_as_int(f[4 * i]), __float_as_int(f[4 * i + 1]),
                                __float_as_int(f[4 * i + 2]), __float_as_int(f[4 * i + 3])));
    } else {
        st_stream((int4 *)p + v, pack8(f));
    }
}

// Eight weights (read again for every row, from L1).
__device__ __forceinline__ void load_weight(const void *w, bool f32, int v, float (&f)[8])
{
    if (f32) {
        const float4 a = __ldg((const float4 *)w + 2 * v), b = __ldg((const float4 *)w + 2 * v + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(__ldg((const int4 *)w + v), f);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// The team's sums of COUNT values, the same for all of its threads.  `turn` alternates
// between a CTA's rows, so that one barrier a row is enough.
template <int WARPS, int COUNT>
__device__ __forceinline__ void team_sum(float (&v)[COUNT], int turn)
{
#pragma unroll
    for (int c = 0; c < COUNT; c++) v[c] = warp_sum(v[c]);
    if constexpr (WARPS > 1) {
        __shared__ float part[2][COUNT][kTeams<WARPS>][WARPS];
        const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * WARPS), warp = threadIdx.x / 32 % WARPS;
#pragma unroll
        for (int c = 0; c < COUNT; c++)
            if (lane == 0) part[turn][c][team][warp] = v[c];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * WARPS) : "memory");
#pragma unroll
        for (int c = 0; c < COUNT; c++) {
            if constexpr (WARPS <= 4) {
                v[c] = part[turn][c][team][0];
#pragma unroll
                for (int w = 1; w < WARPS; w++) v[c] += part[turn][c][team][w];
            } else {
                v[c] = warp_sum(lane < WARPS ? part[turn][c][team][lane] : 0.f);
            }
        }
    }
}

// Values are divided by 2^8 before they are squared: 2^16 / H of the sum is at least 2, so it leaves fp32 only
// where the mean square does.  That changes no bit of it but where squares fall below fp32's normal range, by
// at most 2^-134 of the mean square, which an eps of 2^-100 or more does not see.  (A constant: as an argument
// it took the gradient of 9,000 rows of 6,000 from 77 to 82 us, rows taken again where the sum is infinite to 89.)
constexpr float kSquareScale = 1.f / 256, kSquareUnit = 65536.f;

struct NormArgs {
    const int4 *x;
    const void *residual, *weight;
    bool weight_f32;
    int64_t rows;
    int V;                       // vectors of a row
    float by, eps;               // kSquareUnit / H
    void *residual_out;
    int4 *y;
    uint8_t *record;
};

template <int NV, int WARPS, bool F32>
__global__ void __launch_bounds__(kThreads<WARPS>) k_rms_norm(const __grid_constant__ NormArgs p)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kTeam = 32 * WARPS;
    const int t = threadIdx.x % kTeam;
    const int record_bytes = 8 * p.V + p.V / 4;
    const int64_t r = (int64_t)blockIdx.x * kTeams<WARPS> + threadIdx.x / kTeam;
    if (r < p.rows) {
        int4 x[NV];
        Raw8<F32> res[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            x[i] = make_int4(0, 0, 0, 0);
            if (v < p.V) x[i] = ld_stream(p.x + r * p.V + v);
            res[i].zero();
            if (p.residual && v < p.V) res[i].load(p.residual, r * p.V + v);
        }
        float h[NV][8], sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float add[8];
            unpack8(x[i], h[i]);
            res[i].values(add);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (p.residual) h[i][j] += add[j];      // (-0 stays -0 without a residual)
                const float small = h[i][j] * kSquareScale;
                sum[0] = fmaf(small, small, sum[0]);
            }
            const int v = t + i * kTeam;
            if (p.residual_out && v < p.V) store8<F32>(p.residual_out, r * p.V + v, h[i]);
        }
        team_sum<WARPS, 1>(sum, 0);
        const float inv = 1.f / sqrtf(fmaf(sum[0], p.by, p.eps));
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            float w[8] = {};
            if (v < p.V) load_weight(p.weight, p.weight_f32, v, w);
#pragma unroll
            for (int j = 0; j < 8; j++) w[j] *= h[i][j] * inv;
            const int4 out = pack8(w);
            if (p.y && v < p.V) st_stream(p.y + r * p.V + v, out);
            if (p.record) {                             // whole warps: shuffles
                uint2 code;
                uint8_t scale;
                mxfp8_quantize(out, code, scale);
                uint8_t *to = p.record + r * record_bytes;
                if (v < p.V) {
                    if (record_bytes % 8 == 0) {
                        *(uint2 *)(to + 8 * v) = code;
                    } else {
#pragma unroll
                        for (int b = 0; b < 8; b++)
                            to[8 * v + b] = (uint8_t)((b < 4 ? code.x : code.y) >> (8 * (b & 3)));
                    }
                    if (v % 4 == 0) to[8 * p.V + v / 4] = scale;
                }
            }
        }
    }
}

struct NormBackArgs {
    const int4 *d_y;
    const void *h, *weight, *d_residual;
    bool weight_f32;
    int64_t rows;
    int V;
    float by, eps;
    void *d_h;
    int4 *d_x;
    float *parts;                // [CTAs][8 V], or null: d_w is not wanted
    float by_width;              // 1 / H
};

// The vectors of a row that a thread works on come through shared memory, `AHEAD` rows of
// them: copies of the next rows are under way while a row is summed and written (a thread reads
// what it has copied itself, so its own wait is enough).  AHEAD 0: rows too wide for that,
// straight into registers.
template <int NV, bool F32>
constexpr int kRowSlots = NV * (F32 ? 5 : 3);          // 16 bytes of d_y, h and d_residual each
template <int NV, int WARPS, bool F32, int AHEAD>
constexpr size_t kRingBytes = (size_t)AHEAD * kRowSlots<NV, F32> * kThreads<WARPS> * 16;
// After the last row the teams of a CTA add up their parts of d_w in the same memory.
template <int NV, int WARPS>
constexpr size_t kMergeBytes = kTeams<WARPS> > 1 ? (size_t)NV * 8 * kThreads<WARPS> * 4 : 0;

// (By way of L1: the two halves of a thread's 32 bytes of fp32 are copies of their own, and past L1 each
// fetches the whole sector.  16,384 rows of 5,120 in fp32: 198 us, 265 without; in bf16 105 and 113.)
__device__ __forceinline__ void copy_ahead(int4 *to, const int4 *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
                 : "memory");
}

// CTAs that an SM has registers for at least: two of bf16 rows in small teams (16,384 rows of 5,120: 104 us,
// 111 with one).  Of fp32 rows there are as many as the registers come to, three in the forms of one vector, two
// in small teams of two vectors, but one in teams of ten warps: the rings of two leave L1 too little for the
// second halves of sectors (16,384 rows of 5,120: 266 us, 198 with one), which the grid sees to.
template <int WARPS, bool F32>
constexpr int kCtas = WARPS >= 16 || F32 ? 1 : 2;
template <int WARPS, bool F32>
constexpr bool kOneCta = F32 && WARPS == 10;

template <int NV, int WARPS, bool F32, int AHEAD>
__global__ void __launch_bounds__(kThreads<WARPS>, kCtas<WARPS, F32>)
    k_rms_norm_backward(const __grid_constant__ NormBackArgs p)
{
    extern __shared__ int4 ring[];
    pdl_wait();
    pdl_trigger();
    constexpr int kTeam = 32 * WARPS, kWords = F32 ? 2 : 1, kSlots = kRowSlots<NV, F32>;
    const int t = threadIdx.x % kTeam;
    const int64_t step = (int64_t)gridDim.x * kTeams<WARPS>;
    int64_t r = (int64_t)blockIdx.x * kTeams<WARPS> + threadIdx.x / kTeam;
    auto slot = [&](int stage, int s) { return ring + (stage * kSlots + s) * kThreads<WARPS> + threadIdx.x; };
    auto fetch = [&](int stage, int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            if (row < p.rows && v < p.V) {
                copy_ahead(slot(stage, i), p.d_y + row * p.V + v);
#pragma unroll
                for (int q = 0; q < kWords; q++) {
                    copy_ahead(slot(stage, NV + kWords * i + q), (const int4 *)p.h + (row * p.V + v) * kWords + q);
                    if (p.d_residual)
                        copy_ahead(slot(stage, NV + kWords * (NV + i) + q),
                                   (const int4 *)p.d_residual + (row * p.V + v) * kWords + q);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (AHEAD > 0)
#pragma unroll
        for (int i = 0; i < AHEAD - 1; i++) fetch(i, r + i * step);
    constexpr bool kHold = NV <= 2;                    // weights stay in registers
    float weight[kHold ? NV : 1][8] = {};
    if constexpr (kHold)
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (t + i * kTeam < p.V) load_weight(p.weight, p.weight_f32, t + i * kTeam, weight[i]);
    float acc[NV][8] = {};
    int turn = 0, stage = 0;
    for (; r < p.rows; r += step) {
        float h[NV][8], dy[NV][8], sum[2] = {0.f, 0.f};
        Raw8<F32> res[NV];
        if constexpr (AHEAD > 0) {
            fetch(stage == 0 ? AHEAD - 1 : stage - 1, r + (AHEAD - 1) * step);
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD > 0 ? AHEAD - 1 : 0) : "memory");
        }
        int4 d[NV];
        Raw8<F32> raw[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            d[i] = make_int4(0, 0, 0, 0);
            raw[i].zero();
            res[i].zero();
            if (v < p.V) {
                if constexpr (AHEAD > 0) {
                    d[i] = *slot(stage, i);
#pragma unroll
                    for (int q = 0; q < kWords; q++) raw[i].w[q] = *slot(stage, NV + kWords * i + q);
                } else {
                    d[i] = ld_stream(p.d_y + r * p.V + v);
                    raw[i].load(p.h, r * p.V + v);
                    if (p.d_residual) res[i].load(p.d_residual, r * p.V + v);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            float w[8] = {};
            raw[i].values(h[i]);
            unpack8(d[i], dy[i]);
            if (!kHold && v < p.V) load_weight(p.weight, p.weight_f32, v, w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float small = h[i][j] * kSquareScale;
                sum[0] = fmaf(small, small, sum[0]);
                sum[1] = fmaf(dy[i][j] * (kHold ? weight[i % (kHold ? NV : 1)][j] : w[j]), h[i][j], sum[1]);
            }
        }
        team_sum<WARPS, 2>(sum, turn);
        turn ^= 1;
        const float inv = 1.f / sqrtf(fmaf(sum[0], p.by, p.eps));
        const float along = sum[1] * p.by_width * inv;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            float w[8] = {}, add[8], out[8];
            if (AHEAD > 0 && v < p.V && p.d_residual)
#pragma unroll
                for (int q = 0; q < kWords; q++) res[i].w[q] = *slot(stage, NV + kWords * (NV + i) + q);
            res[i].values(add);
            if (!kHold && v < p.V) load_weight(p.weight, p.weight_f32, v, w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float unit = h[i][j] * inv;
                out[j] = inv * (dy[i][j] * (kHold ? weight[i % (kHold ? NV : 1)][j] : w[j]) - unit * along);
                if (p.d_residual) out[j] += add[j];
                acc[i][j] = fmaf(dy[i][j], unit, acc[i][j]);
            }
            if (v < p.V) {
                store8<F32>(p.d_h, r * p.V + v, out);
                if (p.d_x) st_stream(p.d_x + r * p.V + v, pack8(out));
            }
        }
        if (AHEAD > 0) stage = stage == AHEAD - 1 ? 0 : stage + 1;
    }
    if (!p.parts) return;
    // the CTA's part of d_w: the teams' sums in their order
    if constexpr (kTeams<WARPS> > 1) {
        float *const own = (float *)ring;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) own[(i * 8 + j) * kThreads<WARPS> + threadIdx.x] = acc[i][j];
        __syncthreads();
        for (int at = threadIdx.x; at < NV * 8 * kTeam; at += kThreads<WARPS>) {
            const int column = at / kTeam, u = at % kTeam, v = u + column / 8 * kTeam;
            float s = 0.f;
#pragma unroll
            for (int m = 0; m < kTeams<WARPS>; m++) s += own[column * kThreads<WARPS> + m * kTeam + u];
            if (v < p.V) p.parts[(int64_t)blockIdx.x * 8 * p.V + 8 * v + column % 8] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int v = t + i * kTeam;
            if (v < p.V) {
                float4 *to = (float4 *)(p.parts + (int64_t)blockIdx.x * 8 * p.V) + 2 * v;
                to[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                to[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            }
        }
    }
}

// d_w[c] = the sum of column c over the parts: 32 columns a CTA, its 32 warps take the
// parts in turn, and their sums are added in order.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) k_sum_parts(const float *__restrict__ parts, int count, int H,
                                                           float *__restrict__ d_w)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float own[kSumThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < H)
#pragma unroll 8
        for (int i = warp; i < count; i += kSumThreads / 32) s += __ldcg(parts + (int64_t)i * H + c);
    own[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < H) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kSumThreads / 32; w++) s += own[w][lane];
        d_w[c] = s;
    }
}

template <int NV, int WARPS, bool F32>
cudaError_t norm(const NormArgs &p, cudaStream_t st)
{
    const int64_t grid = (p.rows + kTeams<WARPS> - 1) / kTeams<WARPS>;
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_rms_norm", st,
        err = launch_pdl(k_rms_norm<NV, WARPS, F32>, dim3((unsigned)grid), dim3(kThreads<WARPS>), 0, st, p));
    return err;
}

template <int NV, int WARPS, bool F32>
cudaError_t norm_backward(const NormBackArgs &p, float *d_w, cudaStream_t st)
{
    // Three rows in the ring where two CTAs of them fit an SM, else two (16,384 rows of 5,120: 105 us; past
    // L1, 116 with three rows, 130 with two and 182 straight into registers).  Teams of sixteen warps have
    // an SM's registers to themselves, and take four rows or what its shared memory holds (9,000 rows of
    // 6,000 in fp32: 134 us, 201 straight into registers); with four vectors a thread too that is slower
    // (4,000 rows of 16,000: 148 us for 129).
    constexpr bool kAlone = WARPS >= 16 && NV <= 2;
    constexpr size_t kRoom = kAlone ? 220 * 1024 : 110 * 1024;
    constexpr int kAhead = kAlone && kRingBytes<NV, WARPS, F32, 4> <= kRoom ? 4
                           : kRingBytes<NV, WARPS, F32, 3> <= kRoom         ? 3
                           : kRingBytes<NV, WARPS, F32, 2> <= kRoom         ? 2
                                                                            : 0;
    constexpr size_t kRing = kRingBytes<NV, WARPS, F32, kAhead>, kMerge = kMergeBytes<NV, WARPS>;
    constexpr size_t kSmem = kRing > kMerge ? kRing : kMerge;
    const auto kernel = k_rms_norm_backward<NV, WARPS, F32, kAhead>;
    const int64_t want = (p.rows + kTeams<WARPS> - 1) / kTeams<WARPS>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (err != cudaSuccess) return err;
    int64_t fit = resident_grid((const void *)kernel, kThreads<WARPS>, kSmem);
    if (fit <= 0 || fit > kMaxParts) fit = kMaxParts;
    if (kOneCta<WARPS, F32>) {
        DeviceInfo di;
        err = device_info(&di);
        if (err != cudaSuccess) return err;
        if (fit > di.sm_count) fit = di.sm_count;
    }
    const int64_t grid = want > fit ? fit : want;
    if (grid > 0) {
        MOE_TRACED_LAUNCH("k_rms_norm_backward", st,
            err = launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads<WARPS>), kSmem, st, p));
        if (err != cudaSuccess) return err;
    }
    if (!d_w) return err;
    const int H = 8 * p.V;
    MOE_TRACED_LAUNCH("k_sum_parts", st,
        err = launch_pdl(k_sum_parts, dim3((unsigned)((H + 31) / 32)), dim3(kSumThreads), 0, st,
                         (const float *)p.parts, (int)grid, H, d_w));
    return err;
}

// The team for a row of V vectors: CALL(NV, WARPS).
#define BY_WIDTH(V, CALL)              \
    if ((V) <= 32) return CALL(1, 1);  \
    if ((V) <= 64) return CALL(2, 1);  \
    if ((V) <= 128) return CALL(2, 2); \
    if ((V) <= 192) return CALL(3, 2); \
    if ((V) <= 256) return CALL(2, 4); \
    if ((V) <= 512) return CALL(4, 4); \
    if ((V) <= 640) return CALL(5, 4); \
    if ((V) <= 1024) return CALL(4, 8); \
    if ((V) <= 2048) return CALL(4, 16); \
    return CALL(4, 32)
// Several small teams share a CTA: CTAs of 128 threads start too slowly for short rows (10,525 rows of
// 1,320: 11.7 us, 14.4 with a CTA a row).
// Backward: two vectors a thread where that holds the row, which leaves registers for twenty or
// more warps an SM (16,384 rows of 5,120: 116 us with ten warps and two vectors, 187 with four and five, past L1).
#define BY_WIDTH_BACK(V, CALL)          \
    if ((V) <= 32) return CALL(1, 1);   \
    if ((V) <= 64) return CALL(2, 1);   \
    if ((V) <= 128) return CALL(2, 2);  \
    if ((V) <= 256) return CALL(2, 4);  \
    if ((V) <= 512) return CALL(2, 8);  \
    if ((V) <= 640) return CALL(2, 10); \
    if ((V) <= 1024) return CALL(2, 16); \
    if ((V) <= 2048) return CALL(4, 16); \
    return CALL(4, 32)

}  // namespace

size_t rms_norm_backward_ws_bytes(int64_t rows, int H)
{
    const int64_t parts = rows < 1 ? 1 : rows < kMaxParts ? rows : kMaxParts;
    return ((size_t)parts * H * 4 + 255) / 256 * 256;
}

cudaError_t launch_rms_norm(const uint16_t *x, const void *residual, int residual_type,
                            const void *weight, int weight_type, int64_t rows, int H, float eps,
                            void *residual_out, uint16_t *y, uint8_t *record, cudaStream_t st)
{
    if (rows == 0) return cudaSuccess;
    const NormArgs p{(const int4 *)x, residual, weight, weight_type == MOE_TYPE_F32, rows, H / 8,
                     (float)(1.0 / H) * kSquareUnit, eps, residual_out, (int4 *)y, record};
#define CALL(NV, WARPS) norm<NV, WARPS, true>(p, st)
    if (residual && residual_type == MOE_TYPE_F32) {
        BY_WIDTH(p.V, CALL);
    }
#undef CALL
#define CALL(NV, WARPS) norm<NV, WARPS, false>(p, st)
    BY_WIDTH(p.V, CALL);
#undef CALL
}

cudaError_t launch_rms_norm_backward(const uint16_t *d_y, const void *h, int h_type,
                                     const void *weight, int weight_type, const void *d_residual,
                                     int64_t rows, int H, float eps, void *d_h, uint16_t *d_x,
                                     float *d_weight, void *ws, cudaStream_t st)
{
    const NormBackArgs p{(const int4 *)d_y, h, weight, d_residual, weight_type == MOE_TYPE_F32, rows,
                         H / 8, (float)(1.0 / H) * kSquareUnit, eps, d_h, (int4 *)d_x,
                         d_weight ? (float *)ws : nullptr, (float)(1.0 / H)};
#define CALL(NV, WARPS) norm_backward<NV, WARPS, true>(p, d_weight, st)
    if (h_type == MOE_TYPE_F32) {
        // one vector of 32 bytes a thread (16,384 rows of 2,048: 84 us, 94 with two vectors; 160 and 183 for
        // 4,096).  Rows of bf16 keep two (4,096: 82 us, 90 with one), and so do wider ones (5,120 in fp32: 198
        // us, 305 with one in teams of twenty warps).
        if (p.V > 128 && p.V <= 256) return CALL(1, 8);
        if (p.V > 256 && p.V <= 512) return CALL(1, 16);
        BY_WIDTH_BACK(p.V, CALL);
    }
#undef CALL
#define CALL(NV, WARPS) norm_backward<NV, WARPS, false>(p, d_weight, st)
    BY_WIDTH_BACK(p.V, CALL);
#undef CALL
}

}  // namespace moe
