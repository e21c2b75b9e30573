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
//
// What bounds it: with up to some 80 rows an expert the bytes of the weights in use
// (9/16 byte each), above that the tensor core.  48 rows over 31 of 48 experts of
// 4,096 x 5,120 weights take 62 us, 5.9 TB/s; 16,384 rows over 8 experts of 2,816 x
// 2,048 take 165 to 174 us, 1.1 PFLOP/s.  About 10 us of a call are its start (row counts,
// first rows, first weights: 7 us before the first MMA) and its end.
#include <cuda_bf16.h>
#include <float.h>

#include "common.cuh"
#include "gate.cuh"
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
    const int tiles = w4_tiles(N, gated), chunks = w4_chunks(K), blocks = w4_blocks(N, gated);
    const int64_t pieces = (int64_t)E * tiles * chunks * blocks * (kW4Tile * 4);
    const int rows = gated ? 2 * N : N;
    for (int64_t at = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; at < pieces;
         at += (int64_t)gridDim.x * kPackThreads) {
        // the four pieces of a row are neighbours, so a warp reads whole 64-byte spans
        const int j = (int)(at & 3), i = (int)(at >> 2) & (kW4Tile - 1);
        const int64_t block = at / (kW4Tile * 4);
        const int h = (int)(block % blocks);
        const int c = (int)(block / blocks % chunks);
        const int t = (int)(block / blocks / chunks % tiles);
        const int e = (int)(block / blocks / chunks / tiles);
        const int output = w4_output(t, h, i, N, gated);
        const int n = output < N ? output + (gated && h ? N : 0) : -1;
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
constexpr int kRowsUnseen = 512;    // rows that are read before it is known whether they are used
constexpr int kRowsCtas = 8;        // CTAs per SM
// A row per CTA, or where `a` has more rows than kRowsWide (in use or not) one per warp, which keeps more bytes
// in flight (16,384 rows of 2,048: 24 us by warps, 35 by CTAs) but takes longer for one.
constexpr int kRowsWide = 4096;

// Operand layout of the rows: chunk c of group g at (c * groups + g) * 2048 bytes,
// so a tile's rows are one bulk copy per chunk; in each of its two 64-column
// atoms row r % 8 has 128 bytes, their 16-byte pieces XOR-ed by r % 8.
__device__ __forceinline__ int4 *row_piece(uint8_t *x16, int64_t groups, int64_t group, int r8, int u)
{
    return (int4 *)(x16 + ((u >> 4) * groups + group) * 2048 + (u >> 3 & 1) * 1024 + r8 * 128 +
                    (((u & 7) ^ r8) << 4));
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

// The expert whose run holds row r: the last e < E with offsets[e] <= r, by a warp in
// two ballots over at most 32 values each (E <= 1024).
__device__ __forceinline__ int run_of(const int32_t *offsets, int E, int r)
{
    const int lane = threadIdx.x & 31;
    const int step = (E + 31) / 32;
    const int s = lane * step < E ? __ldg(offsets + lane * step) : 0x7fffffff;
    const unsigned below = __ballot_sync(kFull, s <= r);
    const int base = below ? (31 - __clz((int)below)) * step : 0;
    const int s2 = lane < step && base + lane < E ? __ldg(offsets + base + lane) : 0x7fffffff;
    const unsigned below2 = __ballot_sync(kFull, s2 <= r);
    return base + (below2 ? 31 - __clz((int)below2) : 0);
}

// TEAM threads per row: the CTA's, or a warp's.  With blocks, candidate q is row q / E
// of block q % E, so that the rows in use come first; every warp looks 32 candidates
// over at once.  Also zeroes the arrival counters of k_expert_w4.
template <int TEAM>
__global__ void __launch_bounds__(kRowsThreads, kRowsCtas) k_w4_rows(
    const int4 *__restrict__ a, int a_rows, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ counts, int block_rows, int E, int K, uint8_t *__restrict__ x16,
    float *__restrict__ row_scale, int32_t *__restrict__ arrivals, int n_arrivals)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kHeld = TEAM == 32 ? 8 : 4;       // vectors of a row that a thread keeps
    __shared__ uint32_t part[kRowsThreads / 32];
    const int lane = threadIdx.x & 31, tid = threadIdx.x % TEAM;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_arrivals; i += kRowsThreads) arrivals[i] = 0;
    const int V = K / 8, padded = 16 * w4_chunks(K);
    const int64_t groups = row_groups(a_rows, E);
    const int candidates = offsets ? a_rows : E * block_rows;
    // rows past every run are not read, unless they are few: a load less to wait for
    int end = candidates;
    if (offsets && a_rows > kRowsUnseen) {
        int most = 0;
        for (int i = lane; i <= E; i += 32) most = max(most, __ldg(offsets + i));
        end = min(a_rows, __reduce_max_sync(kFull, most));
    }
    constexpr int kTeamsHere = kRowsThreads / TEAM;
    const int64_t stride = (int64_t)gridDim.x * kTeamsHere;
    for (int64_t q0 = (int64_t)blockIdx.x * kTeamsHere + threadIdx.x / TEAM; q0 < end; q0 += 32 * stride) {
        const int64_t mine = q0 + lane * stride;
        unsigned used = __ballot_sync(kFull, mine < end && (offsets || (int)mine / E <
                                                                           __ldg(counts + (int)mine % E)));
        for (; used; used &= used - 1) {
            const int q = (int)(q0 + (__ffs(used) - 1) * stride);
            const int at = offsets ? q : q % E * block_rows + q / E;
            const int4 *src = a + (int64_t)at * V;
            int4 x[kHeld];                          // the row's first vectors
#pragma unroll
            for (int h = 0; h < kHeld; h++)
                x[h] = tid + h * TEAM < V ? src[tid + h * TEAM] : make_int4(0, 0, 0, 0);
            const int e = offsets ? run_of(offsets, E, q) : q % E;
            int start, count;
            bool bad = false;
            expert_rows(offsets, counts, block_rows, a_rows, e, start, count, bad);
            const int i = at - start;
            if (i < 0 || i >= count) continue;      // uniform per team
            const int64_t group = row_group(offsets != nullptr, start, block_rows, e) + (i >> 3);
            const int r8 = i & 7;
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < kHeld; h++) top = max(top, abs_max_bits(x[h]));
#pragma unroll 4
            for (int v = tid + kHeld * TEAM; v < V; v += TEAM) top = max(top, abs_max_bits(src[v]));
            top = __reduce_max_sync(kFull, top);
            if constexpr (TEAM > 32) {
                __syncthreads();                    // the last row's reads of part[] are over
                if (lane == 0) part[tid >> 5] = top;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < TEAM / 32; w++) top = max(top, part[w]);
            }
            // 2^shift takes the largest value to [2^14, 2^15); at most 2^127 (rows of
            // bf16's smallest values stay below, where fp16 still holds all their bits)
            const int field = (int)(top >> 7);
            const int shift = min(14 - ((field > 0 ? field : 1) - 127), 127);
            const float by = __uint_as_float((uint32_t)(shift + 127) << 23);
            if (tid == 0)
                row_scale[group * 8 + r8] =
                    __uint_as_float(shift == 127 ? 0x00400000u : (uint32_t)(127 - shift) << 23);
            int v = tid;
#pragma unroll
            for (int h = 0; h < kHeld; h++, v += TEAM)
                if (v < padded)
                    st_cg(row_piece(x16, groups, group, r8, v),
                          v < V ? scale_to_half8(x[h], by) : make_int4(0, 0, 0, 0));
            for (; v < padded; v += TEAM)           // (from L1 this time)
                st_cg(row_piece(x16, groups, group, r8, v),
                      v < V ? scale_to_half8(src[v], by) : make_int4(0, 0, 0, 0));
        }
    }
}

// ---------------------------------------------------------------- the product

constexpr int kAStages = 4;                         // decoded blocks in tensor memory
constexpr int kTeams = 3;                           // teams of four warps that decode
constexpr int kDecodeWarps = 4 * kTeams;
constexpr int kEpilogueWarps = 4;
constexpr int kWarpW = kDecodeWarps + kEpilogueWarps, kWarpX = kWarpW + 1, kWarpMma = kWarpW + 2;
constexpr int kMmThreads = (kWarpMma + 1) * 32;     // the last three: weight loads, row loads, MMA
constexpr int kMaxRowsTile = 128;                   // rows of `a` per tile
constexpr int kWStages = 11;                        // 9 KiB weight blocks in flight (18: slower, the
                                                    // first rows come later through the weights)
constexpr int kXBytes = 96 * 1024;                  // ring of row operands
constexpr int kXStagesMax = 12;
constexpr int kAColumns = kW4Chunk / 2;             // 64 columns a block
constexpr int kAFirst = 2 * kMaxRowsTile;           // after the sums
constexpr int kTmemColumns = kAFirst + kAStages * kAColumns;   // 512: all of it
constexpr int64_t kPart = 2 * kMaxRowsTile * kW4Tile;   // partial sums of one part of a tile
constexpr int kMinPart = 12;                        // chunks worth a part of their own
constexpr int kGroupBytes = kW4Chunk / 64 * 1024;   // an 8-row group's chunk: 2 KiB

// A barrier wait tells a phase from the one two before it only by the order of
// events.  A team that waits for weight block j has seen the MMAs of block
// j - kTeams - kAStages end, so a weight stage must come round no sooner than that.
static_assert(kWStages >= kTeams + kAStages, "weight stages come round too soon for the teams' waits");

struct MmShared {
    uint64_t w_full[kWStages], w_empty[kWStages];
    uint64_t x_full[kXStagesMax], x_empty[kXStagesMax];
    uint64_t a_full[kAStages], a_empty[kAStages];
    uint64_t sums_full[2], sums_empty[2];
    int before[kMaxE + 1];           // row tiles of the experts before e
    int start[kMaxE], count[kMaxE];
    uint64_t done;
    uint32_t tmem;
    int most;                        // largest row tile, in 8-row groups
    int total, parts;                // chunks of the call, CTAs that share them
    int base, more;                  // the first `more` CTAs have base + 1 chunks, the rest base
    int last;                        // this CTA arrived last at a cut tile
    volatile int dead;               // a wait gave up
};
constexpr size_t kMmSmem = 1024 + kXBytes + (size_t)kWStages * kW4BlockBytes + sizeof(MmShared);

// Rows per tile: the count in equal parts of at most 128, in MMA steps of 16.
__device__ __forceinline__ int tiles_of(int count) { return (count + kMaxRowsTile - 1) / kMaxRowsTile; }
__device__ __forceinline__ int rows_per_tile(int count, int tiles)
{
    return ((tiles == 1 ? count : (count + tiles - 1) / tiles) + 15) / 16 * 16;
}

struct Segment {
    int e, tile, row0, rows;         // expert, weight tile, rows of `a` in the tile
    int c0, c1;                      // chunks of the segment
    int task;
};

// The last e < E with before[e] * tiles <= task, by a whole warp: two ballots over
// at most 32 values each (E <= 1024).
__device__ __forceinline__ int expert_of(const MmShared &sh, int E, int tiles, int task)
{
    const int lane = threadIdx.x & 31;
    const int step = (E + 31) / 32;
    const int at = lane * step;
    const unsigned below = __ballot_sync(kFull, at < E && sh.before[at] * tiles <= task);
    const int base = (31 - __clz((int)below)) * step;      // before[0] = 0: some bit is set
    if (step == 1) return base;
    const unsigned below2 =
        __ballot_sync(kFull, lane < step && base + lane < E && sh.before[base + lane] * tiles <= task);
    return base + 31 - __clz((int)below2);
}

struct WorkShape {
    int E, tiles, chunks, blocks;
};

// The chunk that CTA b starts with, and the CTA that has chunk g.
__device__ __forceinline__ int first_chunk(const MmShared &sh, int b) { return b * sh.base + min(b, sh.more); }
__device__ __forceinline__ int owner_of(const MmShared &sh, int g)
{
    const int longer = sh.more * (sh.base + 1);
    return g < longer ? g / (sh.base + 1) : sh.more + (g - longer) / sh.base;
}

// The chunks of this CTA, one tile after the other; for whole warps.
struct Walk {
    const MmShared &sh;
    const WorkShape &w;
    int at, to;
    int task, c0;
    __device__ Walk(const MmShared &s, const WorkShape &shape) : sh(s), w(shape)
    {
        const int b = blockIdx.x;
        at = b < sh.parts ? first_chunk(sh, b) : 0;
        to = b < sh.parts ? first_chunk(sh, b + 1) : 0;
        task = at / w.chunks;
        c0 = at - task * w.chunks;
    }
    __device__ bool next(Segment &g)
    {
        if (at >= to) return false;
        g.task = task;
        g.c0 = c0;
        g.c1 = min(w.chunks, c0 + to - at);
        at += g.c1 - g.c0;
        task++;
        c0 = 0;
        g.e = expert_of(sh, w.E, w.tiles, g.task);
        const int local = g.task - sh.before[g.e] * w.tiles;
        const int nt = sh.before[g.e + 1] - sh.before[g.e];
        const int count = sh.count[g.e];
        if (nt == 1) {
            g.tile = local;
            g.row0 = 0;
            g.rows = count;
        } else {
            const int per = rows_per_tile(count, nt);
            g.tile = local / nt;
            g.row0 = (local - g.tile * nt) * per;
            g.rows = min(per, count - g.row0);
        }
        return true;
    }
};

// Parts of a tile that are in memory, and with them their sums.
__device__ __forceinline__ int arrived(const int32_t *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// After a wait that gave up: waits (with a limit) for the copies in flight, whose
// barriers are `full`; `next` is the stage to be filled next, in phase `phase`.
__device__ __forceinline__ void drain(uint64_t *full, int stages, int next, uint32_t phase,
                                      uint32_t issued)
{
    for (int i = 0; i < stages; i++)
        for (int n = 0; (issued >> i & 1) && n < 100000; n++)
            if (mbar_try(&full[i], i < next ? phase : phase ^ 1)) break;
}

// One block times one chunk of rows: eight steps of 16 columns, 32 bytes apart in an
// atom of the row operand, the atoms 1 KiB.
__device__ __forceinline__ void mma_block(uint32_t sums, uint32_t a, uint64_t b, uint32_t word, bool add)
{
#pragma unroll
    for (int i = 0; i < kW4Chunk / 16; i++)
        mma_f16(sums, a + i * 8, b + (uint64_t)((i & 3) * 2 + (i >> 2) * 64), word, add || i > 0);
}

struct Finish {
    uint32_t sums;             // the tile's sums in tensor memory, at this warp's lanes
    int second;                // columns from the first block's sums to the second's
    const float *from;         // parts of a cut tile: at this thread's row of the first one
    int parts, here;           // how many, and which of them is in tensor memory only (-1: none)
    bool have;                 // two parts, the first eight columns of the other are loaded already
    float f;
    int rows;                  // rows of `a`
    int team, teams;           // the teams that finish the tile take its rows of `a` in turn
};

// Sums of COLS rows of `a` from c0 on, for BLOCKS blocks from h on, times the rows'
// scales and the expert's factor; of a cut tile (CUT) over all of its parts in
// their order.
template <int COLS, int BLOCKS, bool CUT>
__device__ __forceinline__ void tile_sums(const Finish &p, int h, int c0,
                                          const float (&scale)[kMaxRowsTile / 32],
                                          const float (&ahead)[2][8], float (&v)[BLOCKS][COLS])
{
    if (!CUT || p.here >= 0)
#pragma unroll
        for (int b = 0; b < BLOCKS; b++) tmem_load(p.sums + (h + b) * p.second + c0, v[b]);
    if constexpr (CUT) {
        if (p.have && c0 == 0) {
#pragma unroll
            for (int b = 0; b < BLOCKS; b++)
#pragma unroll
                for (int j = 0; j < COLS; j++)
                    v[b][j] = 0.f + v[b][j] + (h + b ? ahead[1][j] : ahead[0][j]);
        } else {
            float sum[BLOCKS][COLS] = {};
            // a part that starts the tile is its CTA's last, any other its first
            const float *at = p.from + (h * kMaxRowsTile + c0) * kW4Tile;
            for (int q = 0; q < p.parts; q++) {
                const float *part = at + (2 * q + (q == 0)) * kPart;
#pragma unroll
                for (int b = 0; b < BLOCKS; b++)
#pragma unroll
                    for (int j = 0; j < COLS; j++)
                        sum[b][j] += q == p.here
                                         ? v[b][j]
                                         : __ldcg(part + (b * kMaxRowsTile + j) * kW4Tile);
            }
#pragma unroll
            for (int b = 0; b < BLOCKS; b++)
#pragma unroll
                for (int j = 0; j < COLS; j++) v[b][j] = sum[b][j];
        }
    }
    const float mine = c0 < 32 ? scale[0] : c0 < 64 ? scale[1] : c0 < 96 ? scale[2] : scale[3];
#pragma unroll
    for (int j = 0; j < COLS; j++) {
        const float by = __shfl_sync(kFull, mine, (c0 + j) & 31);
#pragma unroll
        for (int b = 0; b < BLOCKS; b++) v[b][j] = v[b][j] * p.f * by;   // (by alone could overflow)
    }
}

// Outputs of this thread's weight row(s), COLS rows of `a` at a time.  dst: the
// output of the tile's first row of `a`; `store`: not padding.
template <int COLS, bool CUT>
__device__ __forceinline__ void finish_gated(const Finish &p, const float (&scale)[kMaxRowsTile / 32],
                                             const float (&ahead)[2][8], __nv_bfloat16 *dst, int N,
                                             bool store)
{
#pragma unroll 1
    for (int c0 = p.team * COLS; c0 < p.rows; c0 += p.teams * COLS) {
        float v[2][COLS];
        tile_sums<COLS, 2, CUT>(p, 0, c0, scale, ahead, v);
        if (store)
#pragma unroll
            for (int j = 0; j < COLS; j++)
                if (c0 + j < p.rows)
                    dst[(int64_t)(c0 + j) * N] = __float2bfloat16_rn(gated_output(v[0][j], v[1][j]));
    }
}
template <int COLS, bool CUT>
__device__ __forceinline__ void finish_plain(const Finish &p, int h,
                                             const float (&scale)[kMaxRowsTile / 32],
                                             const float (&ahead)[2][8], __nv_bfloat16 *dst, int N,
                                             bool store)
{
#pragma unroll 1
    for (int c0 = p.team * COLS; c0 < p.rows; c0 += p.teams * COLS) {
        float v[1][COLS];
        tile_sums<COLS, 1, CUT>(p, h, c0, scale, ahead, v);
        if (store)
#pragma unroll
            for (int j = 0; j < COLS; j++)
                if (c0 + j < p.rows) dst[(int64_t)(c0 + j) * N] = __float2bfloat16_rn(v[0][j]);
    }
}

// By one warp: the experts' rows, and before[e], the row tiles of those before e.
// Runs could only overlap where the offsets fall: from there on no expert has rows.
__device__ __forceinline__ void scan_experts(MmShared &sh, const int32_t *offsets,
                                             const int32_t *counts, int block_rows, int a_rows,
                                             const WorkShape &w, uint32_t *dev_status)
{
    const int E = w.E;
    constexpr int kAhead = 4;            // loads in flight
    const int lane = threadIdx.x & 31;
    int tiles_before = 0, most = 0;
    bool fell = false, bad = false;
    for (int e0 = 0; e0 < E; e0 += 32 * kAhead) {
        int start[kAhead], count[kAhead];
        bool falls[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int e = e0 + 32 * i + lane;
            start[i] = count[i] = 0;
            falls[i] = false;
            if (e < E) {
                expert_rows(offsets, counts, block_rows, a_rows, e, start[i], count[i], bad);
                falls[i] = offsets && __ldg(offsets + e + 1) < __ldg(offsets + e);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int e = e0 + 32 * i + lane;
            if (e0 + 32 * i >= E) break;
            const unsigned fall = __ballot_sync(kFull, falls[i]);
            if (fell || (fall & (lanemask_lt() | 1u << lane))) count[i] = 0;
            fell = fell || fall;
            const int n = tiles_of(count[i]);
            if (n > 0) most = max(most, rows_per_tile(count[i], n) / 8);
            const int inc = warp_inclusive_scan(n);
            if (e < E) {
                sh.start[e] = start[i];
                sh.count[e] = count[i];
                sh.before[e] = tiles_before + inc - n;
            }
            tiles_before += __shfl_sync(kFull, inc, 31);
        }
    }
    most = __reduce_max_sync(kFull, most);
    if (lane == 0) {
        sh.before[E] = tiles_before;
        sh.most = most;
        // Every CTA takes part where that leaves it kMinPart chunks; else the tiles are cut
        // into parts of at least that (short tiles not at all).
        const int tasks = tiles_before * w.tiles, total = tasks * w.chunks;
        const int most_parts = max(1, w.chunks / kMinPart);
        const int parts = tasks * most_parts <= (int)gridDim.x ? tasks * most_parts
                                                               : min(total, (int)gridDim.x);
        sh.total = total;
        sh.parts = parts;
        sh.base = parts ? total / parts : 0;
        sh.more = parts ? total - sh.base * parts : 0;
        const int warps = (w.blocks == 2 && most > 8 ? kDecodeWarps : 0) + kEpilogueWarps;
        mbar_init(&sh.sums_empty[0], warps);
        mbar_init(&sh.sums_empty[1], warps);
        mbar_init_fence();
    }
    if (bad && blockIdx.x == 0) flag_status(dev_status, MOE_ERR_INVALID_ARG);
    __syncwarp();
}

// The weight warp's work: the CTA's blocks into the ring.
__device__ __forceinline__ void load_weights(MmShared &sh, uint8_t *wring, const uint8_t *w4,
                                             const WorkShape &w)
{
    Walk walk(sh, w);
    Segment g;
    int s = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
        // (the blocks of a segment are one after the other in memory)
        const uint8_t *src = w4 + (((int64_t)g.e * w.tiles + g.tile) * w.chunks + g.c0) * w.blocks *
                                      (int64_t)kW4BlockBytes;
        for (int i = 0; i < (g.c1 - g.c0) * w.blocks; i++, src += kW4BlockBytes) {
            if (!(ok = mbar_wait_warp(&sh.w_empty[s], phase ^ 1, &sh.dead))) break;
            if (elect_lane()) {
                mbar_expect(&sh.w_full[s], kW4BlockBytes);
                bulk_load(wring + s * kW4BlockBytes, src, kW4BlockBytes, &sh.w_full[s]);
            }
            __syncwarp();
            issued |= 1u << s;
            if (++s == kWStages) {
                s = 0;
                phase ^= 1;
            }
        }
    }
    if (!ok) drain(sh.w_full, kWStages, s, phase, issued);
}

struct MmArgs {
    const uint8_t *w4;
    const float *factor;
    const uint8_t *x16;
    const float *row_scale;
    float *partial;
    int32_t *arrivals;
    const int32_t *offsets, *counts;
    int block_rows, a_rows, E, N, K;
    bool gated;
    __nv_bfloat16 *y;
    uint32_t *dev_status;
};

// One block of a thread's weight row out of shared memory (q, sc) into 64 columns of
// its tensor-memory lane: code times scale, exact in fp16.
__device__ __forceinline__ void decode_block(const uint4 (&q)[4], uint2 sc, uint32_t a_at)
{
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const uint32_t s4 = h ? sc.y : sc.x;
        const uint32_t s01 = e4m3x2_to_half2(s4), s23 = e4m3x2_to_half2(s4 >> 16);
        const uint32_t group_scale[4] = {__byte_perm(s01, 0, 0x1010), __byte_perm(s01, 0, 0x3232),
                                         __byte_perm(s23, 0, 0x1010), __byte_perm(s23, 0, 0x3232)};
        const uint32_t word[8] = {q[2 * h].x,     q[2 * h].y,     q[2 * h].z,     q[2 * h].w,
                                  q[2 * h + 1].x, q[2 * h + 1].y, q[2 * h + 1].z, q[2 * h + 1].w};
        uint32_t out[32];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            uint32_t half2s[4];
            e2m1x8_to_half2(word[i], half2s);
#pragma unroll
            for (int j = 0; j < 4; j++) out[4 * i + j] = mul_half2(half2s[j], group_scale[i >> 1]);
        }
        tmem_store32(a_at + h * 32, out);
    }
    tmem_wait_st();
}

// The end of a segment, by `teams` teams of four warps: waits for its sums (stage d of
// them, at `sums` in this warp's lanes, the second block's `second` columns on) and
// writes the tile's outputs, or this part of a cut tile's sums to memory.  A thread has
// one row of each of the tile's blocks.  (Inlined: as a function of its own it made the
// whole kernel a quarter slower, as does any variant that takes local memory.)
__device__ __forceinline__ bool finish_segment(const MmArgs &p, MmShared &sh, const WorkShape &w, Segment g,
                                            uint32_t sums, int second, int d, uint32_t parity, int team,
                                            int teams, bool ok)
{
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = quarter * 32 + lane;
    // A sum is below 2^47; of a factor above 1 half the power of two goes to the rows' scales
    // (at most 2^114), so that neither product leaves fp32 where the result does not.  (A
    // clamped scale would be that of a row whose results leave fp32, or are 0.)
    float f = __ldg(p.factor + g.e);
    const int field = __float_as_int(f) >> 23 & 255;
    const int half = field > 127 ? (field - 127) >> 1 : 0;
    const float rest = __int_as_float((127 + half) << 23);
    f *= __int_as_float((127 - half) << 23);
    const int64_t scale0 =
        (int64_t)row_group(p.offsets != nullptr, sh.start[g.e], p.block_rows, g.e) * 8 + g.row0;
    __nv_bfloat16 *out = p.y + (int64_t)(sh.start[g.e] + g.row0) * p.N;
    int first = 0, parts = 1;
    if (g.c1 - g.c0 < w.chunks) {
        first = owner_of(sh, g.task * w.chunks);
        parts = owner_of(sh, g.task * w.chunks + w.chunks - 1) - first + 1;
    }
    float scale[kMaxRowsTile / 32];      // of rows lane, lane + 32, ... of the tile
#pragma unroll
    for (int i = 0; i < kMaxRowsTile / 32; i++)
        scale[i] = lane + 32 * i < g.rows
                       ? fminf(__ldcg(p.row_scale + scale0 + lane + 32 * i) * rest, FLT_MAX)
                       : 0.f;
    // where the other part of a tile cut in two is in memory already, its first columns
    const bool early = parts > 1 && arrived(p.arrivals + first) == parts - 1;
    const int other = blockIdx.x == first ? first + 1 : first;
    float ahead[2][8];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int j = 0; j < 8; j++)
            ahead[h][j] = early && parts == 2 && h < w.blocks
                              ? __ldcg(p.partial + (2 * other + (other == first)) * kPart +
                                       (h * kMaxRowsTile + j) * kW4Tile + row)
                              : 0.f;
    // one answer for all the warps, which meet at barriers below
    if (!named_all(1, teams * 128, ok && mbar_wait(&sh.sums_full[d], parity, &sh.dead))) return false;
    tmem_fence_after();
    // a cut tile: its last part to be done is summed here with the others' from memory, any
    // other part goes there
    bool finish = true, held = true;       // held: this part's sums are in tensor memory only
    if (parts > 1 &&
        !(finish = named_all(1, teams * 128, early || arrived(p.arrivals + first) == parts - 1))) {
        held = false;
        float *slot = p.partial + (int64_t)(2 * blockIdx.x + (g.c0 == 0)) * kPart;
        for (int h = 0; h < w.blocks; h++)
            for (int c0 = team * 8; c0 < g.rows; c0 += teams * 8) {
                float v[8];
                tmem_load(sums + h * second + c0, v);
#pragma unroll
                for (int j = 0; j < 8; j++) __stcg(slot + (h * kMaxRowsTile + c0 + j) * kW4Tile + row, v[j]);
            }
        __threadfence();
        named_barrier(1, teams * 128);
        if (team == 0 && row == 0) sh.last = atomicAdd(p.arrivals + first, 1) == parts - 1;
        named_barrier(1, teams * 128);
        finish = sh.last;
        __threadfence();
    }
    if (finish) {
        const Finish fin{sums, second, p.partial + (int64_t)2 * first * kPart + row, parts,
                         held ? (int)blockIdx.x - first : -1, early && parts == 2, f, g.rows, team, teams};
        if (p.gated) {
            const int n = w4_output(g.tile, 0, row, p.N, true);
            if (parts > 1) finish_gated<8, true>(fin, scale, ahead, out + n, p.N, n < p.N);
            else if (g.rows <= 8) finish_gated<8, false>(fin, scale, ahead, out + n, p.N, n < p.N);
            else finish_gated<16, false>(fin, scale, ahead, out + n, p.N, n < p.N);
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (h == w.blocks) break;
                const int n = w4_output(g.tile, h, row, p.N, false);
                if (parts > 1) finish_plain<8, true>(fin, h, scale, ahead, out + n, p.N, n < p.N);
                else if (g.rows <= 8) finish_plain<8, false>(fin, h, scale, ahead, out + n, p.N, n < p.N);
                else finish_plain<16, false>(fin, h, scale, ahead, out + n, p.N, n < p.N);
            }
        }
    }
    tmem_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.sums_empty[d]);
    return true;
}

__global__ void __launch_bounds__(kMmThreads, 1) k_expert_w4(const __grid_constant__ MmArgs p)
{
    extern __shared__ uint8_t raw[];
    uint8_t *xring = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
    uint8_t *wring = xring + kXBytes;
    MmShared &sh = *(MmShared *)(wring + kWStages * kW4BlockBytes);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);
    const int tiles = w4_tiles(p.N, p.gated), chunks = w4_chunks(p.K), blocks = w4_blocks(p.N, p.gated);

    // The row counts are older than k_w4_rows, which has passed its own wait when
    // this kernel starts: they and the weights may be read before pdl_wait.
    pdl_trigger();
    volatile int *dead = &sh.dead;
    const WorkShape shape{p.E, tiles, chunks, blocks};
    if (warp == kWarpW) {
        // ---- weight blocks, one bulk copy each.  This warp first finds out what there is to do,
        // in shared memory for all.
        if (lane < kWStages) {
            mbar_init(&sh.w_full[lane], 1);
            mbar_init(&sh.w_empty[lane], 4);
        }
        if (lane == 0) sh.dead = 0;
        mbar_init_fence();
        scan_experts(sh, p.offsets, p.counts, p.block_rows, p.a_rows, shape, p.dev_status);
        named_barrier(2, kMmThreads);
        load_weights(sh, wring, p.w4, shape);
        __syncthreads();
        return;
    }
    if (warp == kWarpX) {
        if (lane < kXStagesMax) {
            mbar_init(&sh.x_full[lane], 1);
            mbar_init(&sh.x_empty[lane], 1);
        }
        if (lane < kAStages) {
            mbar_init(&sh.a_full[lane], 4);
            mbar_init(&sh.a_empty[lane], 1);
        }
        if (lane < 2) mbar_init(&sh.sums_full[lane], 1);
        if (lane == 2) mbar_init(&sh.done, 1);
        mbar_init_fence();
    } else if (warp == kWarpMma) {
        tmem_alloc(&sh.tmem, kTmemColumns);
        tmem_fence_before();
    }
    named_barrier(2, kMmThreads);
    tmem_fence_after();

    const uint32_t tmem = sh.tmem;
    Walk walk(sh, shape);
    Segment g;
    bool ok = true;
    // a stage of row operands holds two chunks where that leaves three stages or more
    const int tile_bytes = max(1, sh.most) * kGroupBytes;
    const int x_chunks = 6 * tile_bytes <= kXBytes ? 2 : 1;
    const int x_stage_bytes = x_chunks * tile_bytes;
    const int x_stages = min(kXStagesMax, kXBytes / x_stage_bytes);
    // sums: two tiles of 128 columns in turn, the blocks' 64 columns apart in them, which
    // the epilogue warps finish while the next tile is summed; two blocks with more than
    // 64 rows of `a` take all 256 columns, and the decode warps, which then have nothing
    // to decode into, help to finish the tile (16 warps take a quarter of the time of four)
    const bool large = blocks == 2 && sh.most > 8;
    const int sums_stages = large ? 1 : 2;
    const int second = large ? kMaxRowsTile : kMaxRowsTile / 2;
    const bool runs = p.offsets != nullptr;

    if (warp == kWarpX) {
        // ---- row operands: one bulk copy per chunk, one barrier per stage
        pdl_wait();
        const int64_t groups = row_groups(p.a_rows, p.E);
        int s = 0;
        uint32_t phase = 0, issued = 0;
        while (ok && walk.next(g)) {
            const int64_t group0 = row_group(runs, sh.start[g.e], p.block_rows, g.e) + g.row0 / 8;
            const uint32_t bytes = (g.rows + 7) / 8 * kGroupBytes;
            for (int c = g.c0; c < g.c1; c += x_chunks) {
                const int n = min(x_chunks, g.c1 - c);
                if (!(ok = mbar_wait_warp(&sh.x_empty[s], phase ^ 1, dead))) break;
                if (elect_lane()) {
                    mbar_expect(&sh.x_full[s], n * bytes);
                    for (int i = 0; i < n; i++)
                        bulk_load(xring + s * x_stage_bytes + i * tile_bytes,
                                  p.x16 + ((c + i) * groups + group0) * kGroupBytes, bytes,
                                  &sh.x_full[s]);
                }
                __syncwarp();
                issued |= 1u << s;
                if (++s == x_stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) drain(sh.x_full, x_stages, s, phase, issued);
    } else if (warp == kWarpMma) {
        // ---- MMA
        int sx = 0, sa = 0, d = 0;
        uint32_t px = 0, pa = 0, pd = 0;
        while (ok && walk.next(g)) {
            const uint32_t word = mma_f16_word((g.rows + 15) / 16 * 16);
            if (!(ok = mbar_wait_warp(&sh.sums_empty[d], pd ^ 1, dead))) break;
            const uint32_t sums = tmem + d * kMaxRowsTile;
            int left = 0;                // chunks left in the stage of row operands
            uint64_t b = 0;
            for (int c = g.c0; c < g.c1; c++) {
                // (a stage of row operands that has been waited for passes again)
                if (!(ok = mbar_wait3_warp(&sh.a_full[sa], pa, &sh.a_full[sa + blocks - 1], pa,
                                           &sh.x_full[sx], px, dead)))
                    break;
                tmem_fence_after();
                if (left == 0) {
                    left = min(x_chunks, g.c1 - c);
                    b = mma_smem_word(smem_addr(xring) + sx * x_stage_bytes, kGroupBytes);
                }
                const uint32_t a = tmem + kAFirst + sa * kAColumns;
                if (elect_lane()) {
                    mma_block(sums, a, b, word, c > g.c0);
                    mma_commit(&sh.a_empty[sa]);
                    if (blocks == 2) {
                        mma_block(sums + second, a + kAColumns, b, word, c > g.c0);
                        mma_commit(&sh.a_empty[sa + 1]);
                    }
                    if (left == 1) mma_commit(&sh.x_empty[sx]);
                    if (c == g.c1 - 1) mma_commit(&sh.sums_full[d]);
                }
                __syncwarp();
                b += tile_bytes >> 4;
                if (--left == 0 && ++sx == x_stages) {
                    sx = 0;
                    px ^= 1;
                }
                sa += blocks;
                if (sa == kAStages) {
                    sa = 0;
                    pa ^= 1;
                }
            }
            if (++d == sums_stages) {
                d = 0;
                pd ^= 1;
            }
        }
        // the MMAs in flight end before their memory goes
        if (elect_lane()) mma_commit(&sh.done);
        __syncwarp();
        for (int n = 0; n < 100000 && !mbar_try(&sh.done, 0); n++) {}
    } else {
        // ---- decode: team t of four warps (one per quarter of the tensor-memory lanes, a row
        // a lane) has every kTeams-th block.  Then the tile's outputs.
        const bool decodes = warp < kDecodeWarps, finishes = large || !decodes;
        const int quarter = warp & 3, team = decodes || large ? warp >> 2 : 0;
        const int row = quarter * 32 + lane;
        const uint32_t at_lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        int sw = team;               // stage of the team's next block
        uint32_t pw = 0;
        int mine = team, seen = 0;   // that block's number; blocks of the segments so far
        const int blocks_here = (walk.to - walk.at) * blocks;
        int d = 0;
        uint32_t pd = 0;
        while (ok && walk.next(g)) {
            seen += (g.c1 - g.c0) * blocks;
            // of a large tile's successor each team decodes a block before it helps to finish
            // the tile, so that the MMAs go on at once afterwards (16,384 rows: 184 -> 177 us)
            const int until = large ? min(seen + kTeams, blocks_here) : seen;
            for (; decodes && mine < until; mine += kTeams) {
                if (!(ok = mbar_wait_warp(&sh.w_full[sw], pw, dead))) break;
                const uint8_t *block = wring + sw * kW4BlockBytes;
                uint4 q[4];
#pragma unroll
                for (int j = 0; j < 4; j++) q[j] = *(const uint4 *)(block + (j * kW4Tile + row) * 16);
                const uint2 sc = *(const uint2 *)(block + kW4CodeBytes + row * 8);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.w_empty[sw]);
                sw += kTeams;
                if (sw >= kWStages) {
                    sw -= kWStages;
                    pw ^= 1;
                }
                const int sa = mine % kAStages;
                if (!(ok = mbar_wait_warp(&sh.a_empty[sa], (mine / kAStages & 1) ^ 1, dead))) break;
                tmem_fence_after();
                decode_block(q, sc, at_lanes + kAFirst + sa * kAColumns);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.a_full[sa]);
            }
            if (!finishes) continue;
            pdl_wait();          // what k_w4_rows wrote, the cut tiles' parts, and y
            ok = finish_segment(p, sh, shape, g, at_lanes + d * kMaxRowsTile, second, d, pd, team,
                                large ? kTeams + 1 : 1, ok);
            if (++d == sums_stages) {
                d = 0;
                pd ^= 1;
            }
        }
    }
    __syncthreads();
    if (warp == kWarpMma) {
        if (sh.dead && lane == 0) flag_status(p.dev_status, MOE_ERR_TIMEOUT);
        tmem_fence_after();
        tmem_free(tmem, kTmemColumns);
    }
}

}  // namespace

size_t w4_bytes(int E, int N, int K, bool gated)
{
    return (size_t)E * w4_tiles(N, gated) * w4_chunks(K) * w4_blocks(N, gated) * kW4BlockBytes;
}

cudaError_t launch_w4_pack(const uint8_t *codes, const uint8_t *scales, int E, int N, int K,
                           bool gated, uint8_t *w4, cudaStream_t st)
{
    const int64_t pieces = (int64_t)(w4_bytes(E, N, K, gated) / kW4BlockBytes) * (kW4Tile * 4);
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
constexpr int kMaxCtas = 160;
size_t align256(size_t n) { return (n + 255) / 256 * 256; }
size_t x16_bytes(int a_rows, int E, int K)
{
    return align256((size_t)row_groups(a_rows, E) * w4_chunks(K) * kGroupBytes);
}
size_t scale_bytes(int a_rows, int E) { return align256((size_t)row_groups(a_rows, E) * 8 * 4); }
constexpr size_t kPartialBytes = (size_t)2 * kMaxCtas * kPart * 4;

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
    const bool by_warp = a_rows > kRowsWide;
    const int want = by_warp ? (a_rows + kRowsThreads / 32 - 1) / (kRowsThreads / 32) : a_rows;
    const int most = kRowsCtas * di.sm_count;
    MOE_TRACED_LAUNCH("k_w4_rows", st,
        err = launch_pdl(by_warp ? k_w4_rows<32> : k_w4_rows<kRowsThreads>,
                         dim3(want > most ? most : want), dim3(kRowsThreads), 0, st, (const int4 *)a,
                         a_rows, offsets, counts, block_rows, E, K, x16, row_scale, arrivals, kMaxCtas));
    if (err != cudaSuccess) return err;
    err = cudaFuncSetAttribute(k_expert_w4, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMmSmem);
    if (err != cudaSuccess) return err;
    MOE_TRACED_LAUNCH("k_expert_w4", st,
        err = launch_pdl(k_expert_w4, dim3(ctas), dim3(kMmThreads), kMmSmem, st,
                         MmArgs{w4, factor, x16, row_scale, partial, arrivals, offsets, counts,
                                block_rows, a_rows, E, N, K, gated, (__nv_bfloat16 *)y, dev_status}));
    return err;
}

}  // namespace moe
