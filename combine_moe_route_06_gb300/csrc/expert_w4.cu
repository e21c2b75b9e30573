// expert_w4.cu -- the experts' products with 4-bit weights.
//
// y[r] = factor[e] * (a[r] . W_e^T) for the rows r of expert e's run, W_e of
// E2M1 codes with one E4M3 scale per 16 columns; gated: W_e = [gate; up] and
// y[r] = silu(a[r] . gate^T) * (a[r] . up^T).  The layout and the decoding of
// the weights are in w4.cuh.
//
// Two kernels.  k_w4_rows writes the rows of `a` as fp16 with a power-of-two
// scale per row (its largest value lands in [2^14, 2^15), so values down to
// 2^-28 of it keep all bf16 bits and the rest a step of 2^-39 of it), in the
// order in which the tensor core reads them from shared memory.  k_expert_w4
// multiplies: the weights are the 128-row operand of tcgen05.mma, decoded from
// 4 bits into tensor memory (exact in fp16), the rows of `a` its other operand
// from shared memory, the sums fp32 in tensor memory.
//
// The work is a list of chunks (expert, 128-row weight tile, tile of at most
// 128 rows of `a`, 128 columns), cut evenly over the CTAs, one per SM: with few
// rows the weights' bytes are the bound and every SM streams the same number of
// them whatever the expert counts.  A tile cut between CTAs is summed from their
// partial sums, in CTA order, by the one that arrives last.
#include <cuda_bf16.h>

#include "common.cuh"
#include "launch.h"
#include "tensor.cuh"
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

// ---------------------------------------------------------------- rows of `a`

// The rows of expert e take 8-row groups from group row_group(e) on: start/8 + e
// for runs, so that no two experts share a group whatever the counts are.
__device__ __forceinline__ int row_group(bool runs, int start, int block_rows, int e)
{
    return runs ? start / 8 + e : e * ((block_rows + 7) / 8);
}
__host__ __device__ __forceinline__ int64_t row_groups(int a_rows, int E)
{
    return (int64_t)a_rows / 8 + E + 1;
}

constexpr int kRowsThreads = 128;
constexpr int kRowsHeld = 4;        // 16-byte vectors of a row that a thread keeps

// Operand layout of the rows: group g, 64-column atom t at ((g * atoms) + t) * 1024
// bytes; in an atom row r % 8 has 128 bytes, its 16-byte pieces XOR-ed by r % 8.
__device__ __forceinline__ int4 *row_piece(uint8_t *x16, int64_t group, int r8, int atoms, int u)
{
    return (int4 *)(x16 + (group * atoms + (u >> 3)) * 1024 + r8 * 128 + (((u & 7) ^ r8) << 4));
}

__device__ __forceinline__ uint32_t abs_max_bits(int4 v)
{
    const uint32_t u[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) m = max(m, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
    return m;
}

__device__ __forceinline__ int4 scale_to_half8(int4 v, float by)
{
    const uint32_t u[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __half2 p = __floats2half2_rn(__uint_as_float(u[i] << 16) * by,
                                            __uint_as_float(u[i] & 0xffff0000u) * by);
        h[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_int4((int)h[0], (int)h[1], (int)h[2], (int)h[3]);
}

// One CTA per row.  Also zeroes the arrival counters of k_expert_w4.
__global__ void __launch_bounds__(kRowsThreads) k_w4_rows(
    const int4 *__restrict__ a, int a_rows, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ counts, int block_rows, int E, int K, uint8_t *__restrict__ x16,
    float *__restrict__ row_scale, int32_t *__restrict__ arrivals, int n_arrivals)
{
    pdl_wait();
    pdl_trigger();
    __shared__ uint32_t part[kRowsThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    if (blockIdx.x == 0)
        for (int i = tid; i < n_arrivals; i += kRowsThreads) arrivals[i] = 0;
    const int V = K / 8, atoms = 2 * w4_chunks(K);
    for (int r = blockIdx.x; r < a_rows; r += gridDim.x) {
        // the expert whose run or block holds row r
        int e;
        if (offsets) {
            const int step = (E + 31) / 32;
            const int at = lane * step;
            const int s = at < E ? __ldg(offsets + at) : 0x7fffffff;
            const unsigned below = __ballot_sync(kFull, s <= r);
            const int base = below ? (31 - __clz((int)below)) * step : 0;
            const int s2 = lane < step && base + lane < E ? __ldg(offsets + base + lane) : 0x7fffffff;
            const unsigned below2 = __ballot_sync(kFull, s2 <= r);
            e = base + (below2 ? 31 - __clz((int)below2) : 0);
        } else {
            e = r / block_rows;
            if (e >= E) break;          // rows past the last block
        }
        int start, count;
        bool bad = false;
        expert_rows(offsets, counts, block_rows, a_rows, e, start, count, bad);
        const int i = r - start;
        if (i < 0 || i >= count) continue;      // uniform per CTA
        const int64_t group = row_group(offsets != nullptr, start, block_rows, e) + (i >> 3);
        const int r8 = i & 7;
        const int4 *src = a + (int64_t)r * V;
        int4 held[kRowsHeld];
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < kRowsHeld; h++) {
            const int v = tid + h * kRowsThreads;
            held[h] = v < V ? src[v] : make_int4(0, 0, 0, 0);
            top = max(top, abs_max_bits(held[h]));
        }
        for (int v = tid + kRowsHeld * kRowsThreads; v < V; v += kRowsThreads)
            top = max(top, abs_max_bits(src[v]));
        top = __reduce_max_sync(kFull, top);
        __syncthreads();                        // the last row's reads of part[] are over
        if (lane == 0) part[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRowsThreads / 32; w++) top = max(top, part[w]);
        // 2^shift takes the largest value to [2^14, 2^15); at most 2^127 (rows of
        // bf16's smallest values stay below, where fp16 still holds all their bits)
        const int field = (int)(top >> 7);
        const int shift = min(14 - ((field > 0 ? field : 1) - 127), 127);
        const float by = __uint_as_float((uint32_t)(shift + 127) << 23);
        if (tid == 0)
            row_scale[group * 8 + r8] =
                __uint_as_float(shift == 127 ? 0x00400000u : (uint32_t)(127 - shift) << 23);
#pragma unroll
        for (int h = 0; h < kRowsHeld; h++) {
            const int v = tid + h * kRowsThreads;
            if (v < atoms * 8) st_cg(row_piece(x16, group, r8, atoms, v), scale_to_half8(held[h], by));
        }
        for (int v = tid + kRowsHeld * kRowsThreads; v < atoms * 8; v += kRowsThreads)
            st_cg(row_piece(x16, group, r8, atoms, v),
                  v < V ? scale_to_half8(src[v], by) : make_int4(0, 0, 0, 0));
    }
}

// ---------------------------------------------------------------- the product

constexpr int kAStages = 4;                         // decoded blocks in tensor memory
constexpr int kDecodeWarps = 4 * kAStages;          // decode the weights, then the epilogue
constexpr int kMmThreads = (kDecodeWarps + 3) * 32; // + weight loads, row loads, MMA
constexpr int kMaxRowsTile = 128;                   // rows of `a` per tile
constexpr int kWStages = 11;                        // 9 KiB weight blocks in flight
constexpr int kXBytes = 96 * 1024;                  // ring of row operands
constexpr int kXStagesMax = 12;
constexpr int kAColumns = kW4Chunk / 2;             // 64 columns a block
constexpr int kTmemColumns = 512;                   // 128 of sums, 4 x 64 of weights
constexpr int kGroupBytes = kW4Chunk / 64 * 1024;   // an 8-row group's chunk: 2 KiB

struct MmShared {
    uint64_t w_full[kWStages], w_empty[kWStages];
    uint64_t x_full[kXStagesMax], x_empty[kXStagesMax];
    uint64_t a_full[kAStages], a_empty[kAStages];
    uint64_t sums_full;
    int64_t before[kMaxE + 1];       // row tiles of the experts before e
    int start[kMaxE], count[kMaxE];
    float up[kAStages][8][kW4Tile / 2];   // gated epilogue: up factors on their way to the gate's warps
    uint32_t tmem;
    int most;                        // largest row tile, in 8-row groups
    int last;                        // this CTA arrived last at a cut tile
    volatile int dead;               // a wait gave up
};
constexpr size_t kMmSmem = 1024 + kXBytes + (size_t)kWStages * kW4BlockBytes + sizeof(MmShared);

// Rows per tile: the count in equal parts of at most 128, in MMA steps of 16.
__device__ __forceinline__ int tiles_of(int count) { return (count + kMaxRowsTile - 1) / kMaxRowsTile; }
__device__ __forceinline__ int rows_per_tile(int count, int tiles)
{
    return ((count + tiles - 1) / tiles + 15) / 16 * 16;
}

struct Segment {
    int e, tile, row0, rows, n;      // expert, weight tile, rows of `a` in the tile, MMA columns
    int c0, c1;                      // chunks of the segment
    int64_t task;
};

// The chunks [from, to) of this CTA, one tile after the other.
struct Walk {
    const MmShared &sh;
    int64_t at, to;
    int E, tiles, chunks;
    __device__ bool next(Segment &g)
    {
        if (at >= to) return false;
        g.task = at / chunks;
        g.c0 = (int)(at - g.task * chunks);
        const int64_t left = to - at;
        g.c1 = left < chunks - g.c0 ? g.c0 + (int)left : chunks;
        at += g.c1 - g.c0;
        int lo = 0, hi = E - 1;      // the last expert with before[e] * tiles <= task
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sh.before[mid] * tiles <= g.task) lo = mid;
            else hi = mid - 1;
        }
        g.e = lo;
        const int64_t local = g.task - sh.before[lo] * tiles;
        const int nt = (int)(sh.before[lo + 1] - sh.before[lo]);
        g.tile = (int)(local / nt);
        const int part = (int)(local - (int64_t)g.tile * nt);
        const int count = sh.count[lo], per = rows_per_tile(count, nt);
        g.row0 = part * per;
        g.rows = min(per, count - g.row0);
        g.n = (g.rows + 15) / 16 * 16;
        return true;
    }
};

// First chunk of CTA b of B when `total` chunks are cut evenly.
__device__ __forceinline__ int64_t cut(int64_t total, int b, int B) { return total * b / B; }
// The CTA whose part holds chunk g.
__device__ __forceinline__ int owner(int64_t total, int B, int64_t g)
{
    int b = (int)(g * B / total);
    while (cut(total, b + 1, B) <= g) b++;
    while (cut(total, b, B) > g) b--;
    return b;
}

__global__ void __launch_bounds__(kMmThreads, 1) k_expert_w4(
    const uint8_t *__restrict__ w4, const float *__restrict__ factor, const uint8_t *x16,
    const float *row_scale, float *partial, int32_t *arrivals, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ counts, int block_rows, int a_rows, int E, int N, int K, bool gated,
    __nv_bfloat16 *y, uint32_t *dev_status)
{
    extern __shared__ uint8_t raw[];
    uint8_t *xring = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    uint8_t *wring = xring + kXBytes;
    MmShared &sh = *(MmShared *)(wring + kWStages * kW4BlockBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tiles = w4_tiles(N, gated), chunks = w4_chunks(K);

    // The row counts are older than k_w4_rows, which has passed its own wait when
    // this kernel starts: they and the weights may be read before pdl_wait.
    pdl_trigger();
    bool bad = false;
    if (tid == 0) {
        sh.most = 0;
        sh.dead = 0;
        for (int i = 0; i < kWStages; i++) {
            mbar_init(&sh.w_full[i], 1);
            mbar_init(&sh.w_empty[i], 4);
        }
        for (int i = 0; i < kXStagesMax; i++) {
            mbar_init(&sh.x_full[i], 1);
            mbar_init(&sh.x_empty[i], 1);
        }
        for (int i = 0; i < kAStages; i++) {
            mbar_init(&sh.a_full[i], 4);
            mbar_init(&sh.a_empty[i], 1);
        }
        mbar_init(&sh.sums_full, 1);
        mbar_init_fence();
    }
    if (warp == kDecodeWarps + 2) tmem_alloc(&sh.tmem, kTmemColumns);
    __syncthreads();
    int most = 0;
    for (int e = tid; e < E; e += kMmThreads) {
        int start, count;
        expert_rows(offsets, counts, block_rows, a_rows, e, start, count, bad);
        sh.start[e] = start;
        sh.count[e] = count;
        if (count > 0) most = max(most, rows_per_tile(count, tiles_of(count)) / 8);
    }
    if (most > 0) atomicMax(&sh.most, most);
    if (bad && blockIdx.x == 0) flag_status(dev_status, MOE_ERR_INVALID_ARG);
    __syncthreads();
    if (warp == 0) {
        int64_t run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int n = e0 + lane < E ? tiles_of(sh.count[e0 + lane]) : 0;
            int64_t inc = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(kFull, inc, off);
                if (lane >= off) inc += o;
            }
            if (e0 + lane < E) sh.before[e0 + lane] = run + inc - n;
            run += __shfl_sync(kFull, inc, 31);
        }
        if (lane == 0) sh.before[E] = run;
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();

    const uint32_t tmem = sh.tmem;
    const int64_t total = sh.before[E] * tiles * chunks;
    // at least a chunk for every CTA that takes part, so each part of a cut tile arrives
    const int B = total < gridDim.x ? (int)total : gridDim.x;
    const bool idle = (int)blockIdx.x >= B;
    Walk walk{sh, idle ? 0 : cut(total, blockIdx.x, B), idle ? 0 : cut(total, blockIdx.x + 1, B), E,
              tiles, chunks};
    const int x_stages = min(kXStagesMax, kXBytes / max(1, sh.most * kGroupBytes));
    const int x_stage_bytes = sh.most * kGroupBytes;
    volatile int *dead = &sh.dead;
    Segment g;

    if (warp == kDecodeWarps) {
        // ---- weight blocks: one bulk copy each
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            while (ok && walk.next(g)) {
                const uint8_t *src = w4 + (((int64_t)g.e * tiles + g.tile) * chunks + g.c0) *
                                              (int64_t)kW4BlockBytes;
                for (int c = g.c0; c < g.c1; c++, src += kW4BlockBytes) {
                    if (!(ok = mbar_wait(&sh.w_empty[s], phase ^ 1, dead))) break;
                    mbar_expect(&sh.w_full[s], kW4BlockBytes);
                    bulk_load(wring + s * kW4BlockBytes, src, kW4BlockBytes, &sh.w_full[s]);
                    issued |= 1u << s;
                    if (++s == kWStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)            // no copy is left in flight
                for (int i = 0; i < kWStages; i++)
                    if (issued >> i & 1) {
                        const uint32_t last = i < s ? phase : phase ^ 1;
                        for (int n = 0; n < 100000 && !mbar_try(&sh.w_full[i], last); n++) {}
                    }
        }
    } else if (warp == kDecodeWarps + 1) {
        // ---- row operands: one bulk copy per 8-row group
        if (lane == 0) {
            pdl_wait();
            const int atoms = 2 * chunks;
            int s = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            while (ok && walk.next(g)) {
                const int64_t group0 =
                    row_group(offsets != nullptr, sh.start[g.e], block_rows, g.e) + g.row0 / 8;
                const int groups = (g.rows + 7) / 8;
                for (int c = g.c0; c < g.c1; c++) {
                    if (!(ok = mbar_wait(&sh.x_empty[s], phase ^ 1, dead))) break;
                    mbar_expect(&sh.x_full[s], groups * kGroupBytes);
                    uint8_t *dst = xring + s * x_stage_bytes;
                    for (int i = 0; i < groups; i++)
                        bulk_load(dst + i * kGroupBytes,
                                  x16 + ((group0 + i) * atoms + 2 * c) * 1024, kGroupBytes,
                                  &sh.x_full[s]);
                    issued |= 1u << s;
                    if (++s == x_stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)
                for (int i = 0; i < x_stages; i++)
                    if (issued >> i & 1) {
                        const uint32_t last = i < s ? phase : phase ^ 1;
                        for (int n = 0; n < 100000 && !mbar_try(&sh.x_full[i], last); n++) {}
                    }
        }
    } else if (warp == kDecodeWarps + 2) {
        // ---- MMA: eight steps of 16 columns per chunk, issued by one thread
        if (lane == 0) {
            int sx = 0, sa = 0;
            uint32_t px = 0, pa = 0;
            bool ok = true;
            while (ok && walk.next(g)) {
                const uint32_t word = mma_f16_word(g.n);
                for (int c = g.c0; c < g.c1; c++) {
                    if (!(ok = mbar_wait(&sh.x_full[sx], px, dead) &&
                               mbar_wait(&sh.a_full[sa], pa, dead)))
                        break;
                    tmem_fence_after();
                    const uint32_t a = tmem + kMaxRowsTile + sa * kAColumns;
                    const uint64_t b = mma_smem_word(smem_addr(xring) + sx * x_stage_bytes, kGroupBytes);
#pragma unroll
                    for (int i = 0; i < kW4Chunk / 16; i++)     // 32 bytes a step, 1 KiB an atom
                        mma_f16(tmem, a + i * 8, b + (uint64_t)((i & 3) * 2 + (i >> 2) * 64), word,
                                c > g.c0 || i > 0);
                    mma_commit(&sh.a_empty[sa]);
                    mma_commit(&sh.x_empty[sx]);
                    if (++sx == x_stages) {
                        sx = 0;
                        px ^= 1;
                    }
                    if (++sa == kAStages) {
                        sa = 0;
                        pa ^= 1;
                    }
                }
                if (ok) mma_commit(&sh.sums_full);
            }
        }
    } else {
        // ---- decode: team t of four warps (one per quarter of the tensor-memory lanes, a row
        // a lane) has every kAStages-th chunk and A stage t; then the same warps finish the tile
        const int quarter = warp & 3, team = warp >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t a_at = tmem + lanes + kMaxRowsTile + team * kAColumns;
        int sw = team;               // stage of the team's next chunk
        uint32_t pw = 0, pa = 0, psum = 0;
        uint32_t mine = team, seen = 0;      // that chunk's number; chunks of the past segments
        bool ok = true;
        pdl_wait();
        while (ok && walk.next(g)) {
            seen += g.c1 - g.c0;
            for (; mine < seen; mine += kAStages) {
                if (!(ok = mbar_wait(&sh.w_full[sw], pw, dead))) break;
                const uint8_t *block = wring + sw * kW4BlockBytes;
                uint4 q[4];
#pragma unroll
                for (int j = 0; j < 4; j++) q[j] = *(const uint4 *)(block + (j * kW4Tile + row) * 16);
                const uint2 sc = *(const uint2 *)(block + kW4CodeBytes + row * 8);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.w_empty[sw]);
                sw += kAStages;
                if (sw >= kWStages) {
                    sw -= kWStages;
                    pw ^= 1;
                }
                if (!(ok = mbar_wait(&sh.a_empty[team], pa ^ 1, dead))) break;
                pa ^= 1;
                tmem_fence_after();
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint32_t s4 = h ? sc.y : sc.x;
                    const uint32_t s01 = e4m3x2_to_half2(s4), s23 = e4m3x2_to_half2(s4 >> 16);
                    const uint32_t group_scale[4] = {
                        __byte_perm(s01, 0, 0x1010), __byte_perm(s01, 0, 0x3232),
                        __byte_perm(s23, 0, 0x1010), __byte_perm(s23, 0, 0x3232)};
                    const uint32_t word[8] = {q[2 * h].x,     q[2 * h].y,     q[2 * h].z,
                                              q[2 * h].w,     q[2 * h + 1].x, q[2 * h + 1].y,
                                              q[2 * h + 1].z, q[2 * h + 1].w};
                    uint32_t out[32];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        uint32_t half2s[4];
                        e2m1x8_to_half2(word[i], half2s);
#pragma unroll
                        for (int p = 0; p < 4; p++)
                            out[4 * i + p] = mul_half2(half2s[p], group_scale[i >> 1]);
                    }
                    tmem_store32(a_at + h * 32, out);
                }
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.a_full[team]);
            }
            if (!ok || !(ok = mbar_wait(&sh.sums_full, psum, dead))) break;
            psum ^= 1;
            tmem_fence_after();

            // ---- epilogue: a thread has one weight row, eight rows of `a` at a time, the teams
            // in turn
            const int blocks = (g.rows + 7) / 8;
            bool sum_parts = false;
            int first = 0, parts = 1;
            if (g.c1 - g.c0 < chunks) {
                const int64_t task0 = g.task * chunks;
                first = owner(total, B, task0);
                parts = owner(total, B, task0 + chunks - 1) - first + 1;
                float *slot = partial + (int64_t)(2 * blockIdx.x + (g.c0 == 0)) * (kMaxRowsTile * kW4Tile);
                for (int cb = team; cb < blocks; cb += kAStages) {
                    float v[8];
                    tmem_load8(tmem + lanes + cb * 8, v);
#pragma unroll
                    for (int j = 0; j < 8; j++) __stcg(slot + (cb * 8 + j) * kW4Tile + row, v[j]);
                }
                __threadfence();
                named_barrier(1, kDecodeWarps * 32);
                if (tid == 0) sh.last = atomicAdd(arrivals + first, 1) == parts - 1;
                named_barrier(1, kDecodeWarps * 32);
                if (!sh.last) {
                    tmem_fence_before();
                    continue;
                }
                __threadfence();
                sum_parts = true;
            }
            const float f = __ldg(factor + g.e);
            const int64_t scale0 =
                (int64_t)row_group(offsets != nullptr, sh.start[g.e], block_rows, g.e) * 8 + g.row0;
            const int per = w4_outputs_per_tile(gated);
            const int n = g.tile * per + row % per;
            __nv_bfloat16 *dst = y + (int64_t)(sh.start[g.e] + g.row0) * N + n;
            for (int cb = team; cb < blocks; cb += kAStages) {
                float v[8];
                if (sum_parts) {
#pragma unroll
                    for (int j = 0; j < 8; j++) v[j] = 0.f;
                    for (int p = first; p < first + parts; p++) {
                        // a part that starts the tile is its CTA's last, any other its first
                        const float *slot = partial + (int64_t)(2 * p + (p == first)) *
                                                          (kMaxRowsTile * kW4Tile);
#pragma unroll
                        for (int j = 0; j < 8; j++) v[j] += __ldcg(slot + (cb * 8 + j) * kW4Tile + row);
                    }
                } else {
                    tmem_load8(tmem + lanes + cb * 8, v);
                }
#pragma unroll
                for (int j = 0; j < 8; j++)
                    v[j] = v[j] * __ldcg(row_scale + scale0 + cb * 8 + j) * f;
                if (gated) {
                    named_barrier(2 + team, 128);     // the last turn's reads are over
                    if (row >= per)
#pragma unroll
                        for (int j = 0; j < 8; j++) sh.up[team][j][row - per] = v[j];
                    named_barrier(2 + team, 128);
                    if (row < per)
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            v[j] = v[j] / (1.f + __expf(-v[j])) * sh.up[team][j][row];
                }
                if (row < per && n < N)
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (cb * 8 + j < g.rows)
                            dst[(int64_t)(cb * 8 + j) * N] = __float2bfloat16_rn(v[j]);
            }
            tmem_fence_before();
        }
    }
    __syncthreads();
    if (warp == kDecodeWarps + 2) {
        if (sh.dead) {      // MMAs may still run: wait for them before the memory goes
            if (lane == 0) {
                mma_commit(&sh.sums_full);
                flag_status(dev_status, MOE_ERR_TIMEOUT);
            }
            const uint64_t start = global_ns();
            while (global_ns() - start < 1000000ull) {}
        }
        __syncwarp();
        tmem_fence_after();
        tmem_free(tmem, kTmemColumns);
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

namespace {

// Workspace of one call: the rows in operand form, their scales, the partial
// sums of cut tiles (two a CTA) and the arrival counters (one a CTA).
constexpr int kMaxCtas = 256;
size_t align256(size_t n) { return (n + 255) / 256 * 256; }
size_t x16_bytes(int a_rows, int E, int K)
{
    return align256((size_t)row_groups(a_rows, E) * w4_chunks(K) * kGroupBytes);
}
size_t scale_bytes(int a_rows, int E) { return align256((size_t)row_groups(a_rows, E) * 8 * 4); }
constexpr size_t kPartialBytes = (size_t)2 * kMaxCtas * kMaxRowsTile * kW4Tile * 4;

}  // namespace

size_t expert_w4_ws_bytes(int a_rows, int E, int N, int K)
{
    (void)N;
    return x16_bytes(a_rows, E, K) + scale_bytes(a_rows, E) + kPartialBytes + align256(kMaxCtas * 4);
}

cudaError_t launch_expert_w4(const uint16_t *a, int a_rows, const int32_t *offsets,
                             const int32_t *counts, int block_rows, const uint8_t *w4,
                             const float *factor, int E, int N, int K, bool gated, uint16_t *y,
                             void *ws, uint32_t *dev_status, cudaStream_t st)
{
    if (a_rows == 0) return cudaSuccess;
    DeviceInfo di;
    cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    if ((size_t)di.max_smem_optin < kMmSmem) return cudaErrorInvalidConfiguration;
    uint8_t *x16 = (uint8_t *)ws;
    float *row_scale = (float *)(x16 + x16_bytes(a_rows, E, K));
    float *partial = (float *)((uint8_t *)row_scale + scale_bytes(a_rows, E));
    int32_t *arrivals = (int32_t *)((uint8_t *)partial + kPartialBytes);
    const int ctas = di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas;
    const int fit = resident_grid((const void *)k_w4_rows, kRowsThreads, 0);
    const int grid = fit > 0 && a_rows > fit ? fit : a_rows;
    MOE_TRACED_LAUNCH("k_w4_rows", st,
        err = launch_pdl(k_w4_rows, dim3(grid), dim3(kRowsThreads), 0, st, (const int4 *)a, a_rows,
                         offsets, counts, block_rows, E, K, x16, row_scale, arrivals, kMaxCtas));
    if (err != cudaSuccess) return err;
    err = cudaFuncSetAttribute(k_expert_w4, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMmSmem);
    if (err != cudaSuccess) return err;
    MOE_TRACED_LAUNCH("k_expert_w4", st,
        err = launch_pdl(k_expert_w4, dim3(ctas), dim3(kMmThreads), kMmSmem, st, w4, factor,
                         (const uint8_t *)x16, (const float *)row_scale, partial, arrivals, offsets,
                         counts, block_rows, a_rows, E, N, K, gated, (__nv_bfloat16 *)y, dev_status));
    return err;
}

}  // namespace moe
