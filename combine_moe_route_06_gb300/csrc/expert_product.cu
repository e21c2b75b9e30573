// expert_product.cu -- the experts' products with bf16 weights and their gradients.
//
// Three products over the rows of each expert e (W_e [N][K]):
//   y[r][n]   = sum_k a[r][k] W_e[n][k]      (gated: silu of one sum times another)
//   d_a[r][k] = sum_n d_y[r][n] W_e[n][k]    (or, with gate and up, their gradient)
//   d_w[n][k] = sum_r d_y[r][n] a[r][k]
// by one kernel, tcgen05.mma of CTA pairs: D[256][n] += A[256][64] B[n][64]^T a step.
// A is of the weights (for d_w: of d_y, across its rows), B of the rows (for d_w: of a): a
// tile's rows follow the expert's, in steps of 32 up to 256, so that few rows cost few, while
// the weights, which then are the bound, always fill their side.  Each CTA of a pair
// loads half of A and of B by TMA, holds 128 rows of D in tensor memory and finishes them.
// Gated: A has 8 gate rows and the 8 up rows of the same outputs in turn, so that the two
// factors of an output meet in one thread (tmem_load_matrices).
//
// The work is a list of steps (expert, tile, 64 of the summed index).  Where there are many
// tiles the pairs, one per two SMs, take them in turn; the last one or two per pair, or all of
// few, are cut evenly over the pairs: with few rows every SM streams the same number of
// weights.  A tile that is cut is summed from its parts, in pair order, by the one that
// arrives last.
//
// A tensor map fills what lies outside the matrix with zeros, so N and K need no padding;
// rows of B behind an expert's give columns of D that nobody reads.  Only for d_w are rows summed
// over, and those behind the expert's are cleared in shared memory (they may hold anything).
//
// What bounds it: with up to some 290 rows an expert the bytes of the weights in use, above that the
// tensor core.  48 rows over 36 experts of 5,120 x 2,048 take 114 us, 6.6 TB/s; 16,384 rows over 8
// experts of 2,816 x 2,048, gated, 113 us at 1.57 GHz, 1.67 PFLOP/s, the tensor pipe active for 87% of
// it, and 131 us where calls back to back keep the chip at its power limit.  A step's 64 KiB come from L2
// (80% hits: pairs on neighbouring tiles); taken in contiguous ranges of tiles instead, 1.3 GB came from
// HBM and the same call took 236 us.  Shared memory is the other limit: MMA operands and their loads
// take about all of its bandwidth, so what the end of a tile does there counts (stores of single
// values for 8 x 8 matrices: 119 us for 113).
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "gate.cuh"
#include "launch.h"
#include "tensor.cuh"
#include "trace.h"
#include "w4.cuh"

namespace moe {

namespace {

enum Form { kPlain, kGated, kRowGrad, kGateGrad, kWeightGrad };

constexpr int kStep = 64;                        // of the summed index, 128 bytes
constexpr int kTileRows = 256;                   // rows of A and D, most rows of B
constexpr int kStages = 6, kMaxStages = 10;      // of whole tiles, of tiles with few rows on the B side
constexpr int kABytes = 128 * kStep * 2, kBBytes = 128 * kStep * 2, kStageBytes = kABytes + kBBytes;
constexpr int kFinishWarps = 8;
constexpr int kWarpLoad = kFinishWarps, kWarpMma = kFinishWarps + 1, kWarpClear = kFinishWarps + 2;
constexpr int kMmThreads = 32 * (kFinishWarps + 3);
constexpr int kTmemColumns = 512;                // two tiles of 256 columns of sums
constexpr int kSumSteps = 12;                    // d_w: steps summed by the tensor core alone
// Steps worth a part of their own, for tiles of up to 64 rows and of more: the last one reads the sums
// of all (375 rows over 4 experts of 48 x 4,040: 20.8 us with 8 steps, 18.0 with 16).
constexpr int kMinPart = 8, kMinPartWide = 16;
// Steps that the parts of cut tiles take to be joined: where whole tiles leave the pairs waiting for less,
// none is cut (16,384 rows over 8 experts: gated 2,816 x 2,048 125 us with 0, 118 with 24 or more; gradient
// of 1,408 x 2,048 103 us with 0 or 12, 94 with 24, 93 with 40; shorter sums than this are never cut).
constexpr int kCutSteps = 40;
constexpr int64_t kPart = (int64_t)kTileRows * 128;   // sums of one part of a tile, in one CTA
constexpr int kMaxCtas = 160;
constexpr int kCols = 16;                        // columns of D that a warp finishes at once
constexpr int kGroups = kFinishWarps / 4;        // warps that share the columns of 32 rows of D
constexpr int kStaging = 4 * kCols * 32;         // bytes of shared memory a warp has for that

// A tile, or a part of one, that a pair has.
struct Segment {
    int e, tile;                     // expert, tile of the A side
    int row0, rows, cols;            // d_w: first column, columns in the matrix, columns of the MMA;
                                     // else first row of the tile, its rows, and those rounded up
    int c0, c1, steps;               // steps of the segment, of the whole tile
    int unit;                        // first step of the tile
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], landed[kStages], cleared[kStages];
    uint64_t sums_full[2], sums_empty[2];
    int before[kMaxE + 1];           // steps of the experts before e
    int start[kMaxE], count[kMaxE];
    uint32_t tmem;
    int stages, stage_bytes;         // the ring of operands
    int first_pair, pairs;           // the pairs that share the work
    int tasks, waves;                // tiles, and how many of them a pair takes whole, in turn
    int shared;                      // first step of the rest, which is cut evenly
    int parts;                       // pairs that share it
    int base, more;                  // the first `more` pairs have base + 1 steps, the rest base
    int last;
    bool weights;                    // of two products at once this CTA has d_w
    volatile int dead;               // a wait gave up
};
constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kFinishWarps * kStaging + sizeof(Shared);

struct Maps {
    CUtensorMap a, b[3];             // b: boxes of 16, 64 and 128 rows (d_w: the first, of 64)
    CUtensorMap d;                   // d_w
};
struct Args {
    const int32_t *offsets, *counts;
    int block_rows, a_rows, E, N, K;
    int rows_a, sums;                // rows of the A side (outputs of a row), length of the sum
    int most;                        // rows of a tile of the B side: 256, 128 or 64
    __nv_bfloat16 *out, *keep;
    const __nv_bfloat16 *pre;
    bool d_w_f32;
    float *partial;
    int32_t *arrivals;
    uint32_t *dev_status;
};

// Rows of an expert in tiles of at most `most` (a multiple of 32), and where tile i starts: their units of
// 32 in equal parts.
__device__ __forceinline__ int row_tiles(int count, int most) { return (int)(((unsigned)count + most - 1) / most); }
__device__ __forceinline__ int tile_start(int count, int tiles, int i)
{
    return (int)((int64_t)i * (((unsigned)count + 31) / 32) / tiles) * 32;
}

struct Shape {
    int E, tiles;                    // tiles of the A side
    int steps;                       // of a tile (0: by the expert's rows)
    int tiles_b;                     // d_w: tiles of the B side
};

template <int FORM>
__device__ __forceinline__ Shape shape_of(const Args &p)
{
    if (FORM == kWeightGrad)
        return {p.E, (p.N + kTileRows - 1) / kTileRows, 0, (p.K + p.most - 1) / p.most};
    return {p.E, (p.rows_a + kTileRows - 1) / kTileRows, (p.sums + kStep - 1) / kStep, 0};
}
// (an expert without rows has one step, of nothing but the zeros of its gradient)
__device__ __forceinline__ int steps_of(const Shape &w, int count)
{
    return w.steps ? w.steps : max(1, (int)(((unsigned)count + kStep - 1) / kStep));
}

// The steps of this pair, one tile after the other; for whole warps.
template <int FORM>
struct Walk {
    const Shared &sh;
    const Args &p;
    const Shape &w;
    int wave, at, to;
    __device__ Walk(const Shared &s, const Args &a, const Shape &shape) : sh(s), p(a), w(shape)
    {
        const int b = blockIdx.x / 2 - sh.first_pair;
        wave = 0;
        at = sh.shared + (b < sh.parts ? b * sh.base + min(b, sh.more) : 0);
        to = at + (b < sh.parts ? sh.base + (b < sh.more) : 0);
    }
    // The last e with before[e] <= at: two ballots over at most 32 values each (E <= 1024).
    // Experts without steps share their `before` with the next one, which is taken.
    __device__ int expert(int at) const
    {
        const int lane = threadIdx.x & 31, step = (w.E + 31) / 32;
        const unsigned below = __ballot_sync(kFull, lane * step < w.E && sh.before[lane * step] <= at);
        const int base = (31 - __clz((int)below)) * step;         // before[0] = 0: some bit is set
        if (step == 1) return base;
        const unsigned below2 =
            __ballot_sync(kFull, lane < step && base + lane < w.E && sh.before[base + lane] <= at);
        return base + 31 - __clz((int)below2);
    }
    // no segment is left
    __device__ bool over() const
    {
        const int task = wave * sh.pairs + (int)(blockIdx.x / 2) - sh.first_pair;
        return (wave >= sh.waves || task >= sh.tasks) && at >= to;
    }
    __device__ bool next(Segment &g)
    {
        int task, count;
        if (wave < sh.waves) {
            task = wave * sh.pairs + blockIdx.x / 2 - sh.first_pair;
            wave++;
            if (task >= sh.tasks) return false;
            if constexpr (FORM == kWeightGrad) {
                g.e = task / (w.tiles * w.tiles_b);
                task -= g.e * (w.tiles * w.tiles_b);
            } else {
                g.e = expert(task * w.steps);
                task -= sh.before[g.e] / w.steps;
            }
            count = sh.count[g.e];
            g.steps = steps_of(w, count);
            g.c0 = 0;
            g.c1 = g.steps;
            g.unit = 0;
        } else {
            if (at >= to) return false;
            g.e = expert(at);
            count = sh.count[g.e];
            g.steps = steps_of(w, count);
            const int local = at - sh.before[g.e];
            task = local / g.steps;
            g.c0 = local - task * g.steps;
            g.c1 = min(g.steps, g.c0 + to - at);
            g.unit = at - g.c0;
            at += g.c1 - g.c0;
        }
        if constexpr (FORM == kWeightGrad) {
            g.tile = task / w.tiles_b;
            g.row0 = (task - g.tile * w.tiles_b) * p.most;
            g.rows = min(p.most, p.K - g.row0);
        } else {
            const int nt = row_tiles(count, p.most);
            g.tile = task / nt;
            const int i = task - g.tile * nt;
            g.row0 = tile_start(count, nt, i);
            g.rows = min(count, tile_start(count, nt, i + 1)) - g.row0;
        }
        g.cols = (g.rows + 31) / 32 * 32;
        return true;
    }
};
__device__ __forceinline__ int owner_of(const Shared &sh, int unit)
{
    const int longer = sh.more * (sh.base + 1);
    unit -= sh.shared;
    return unit < longer ? unit / (sh.base + 1) : sh.more + (unit - longer) / sh.base;
}

// Rows of B that a CTA loads for `half` rows: by 16 up to 32, else 64 or 128.
__device__ __forceinline__ int loaded_rows(int half) { return half <= 32 ? half : half <= 64 ? 64 : 128; }

// By one warp: the experts' rows, and before[e], the steps of those before e.  Runs could only
// overlap where the offsets fall: from there on no expert has rows.
template <int FORM>
__device__ __forceinline__ void scan_experts(Shared &sh, const Args &p, const Shape &w)
{
    constexpr int kAhead = 4;            // loads in flight
    const int lane = threadIdx.x & 31;
    int before = 0, tasks = 0, longest = 0, widest = 0;
    bool fell = false, bad = false;
    for (int e0 = 0; e0 < p.E; e0 += 32 * kAhead) {
        int start[kAhead], count[kAhead];
        bool falls[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int e = e0 + 32 * i + lane;
            start[i] = count[i] = 0;
            falls[i] = false;
            if (e < p.E) {
                expert_rows(p.offsets, p.counts, p.block_rows, p.a_rows, e, start[i], count[i], bad);
                falls[i] = p.offsets && __ldg(p.offsets + e + 1) < __ldg(p.offsets + e);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int e = e0 + 32 * i + lane;
            if (e0 + 32 * i >= p.E) break;
            const unsigned fall = __ballot_sync(kFull, falls[i]);
            if (fell || (fall & (lanemask_lt() | 1u << lane))) count[i] = 0;
            fell = fell || fall;
            const int n = e >= p.E ? 0 : FORM == kWeightGrad ? w.tiles * w.tiles_b : w.tiles * row_tiles(count[i], p.most);
            const int units = n * steps_of(w, count[i]);
            longest = max(longest, e < p.E ? steps_of(w, count[i]) : 0);
            widest = max(widest, count[i]);
            const int inc = warp_inclusive_scan(units);
            if (e < p.E) {
                sh.start[e] = start[i];
                sh.count[e] = count[i];
                sh.before[e] = before + inc - units;
            }
            before += __shfl_sync(kFull, inc, 31);
            tasks += n;
        }
    }
    tasks = __reduce_add_sync(kFull, tasks);
    longest = __reduce_max_sync(kFull, longest);
    widest = FORM == kWeightGrad ? p.most : min(p.most, __reduce_max_sync(kFull, widest));
    __syncwarp();
    if (lane == 0) {
        sh.before[p.E] = before;
        // Whole tiles in turn, so that the pairs work on neighbouring tiles at the same time, whose
        // operands come from L2.  Cutting the last ones evenly takes kCutSteps, and there is nothing
        // to gain where the pairs' last tiles wait for less; nor are all tiles taken in turn
        // where a few experts have most of the steps.
        const int pairs = sh.pairs, turns = (tasks + pairs - 1) / pairs;
        const bool whole = ((int64_t)turns * pairs - tasks) * longest <= (int64_t)kCutSteps * pairs;
        const bool even = (int64_t)longest * tasks <= 2 * (int64_t)before;
        const int waves = longest <= kCutSteps ? turns : !even ? 0 : whole ? turns : max(0, tasks / pairs - 1);
        const int task = min(tasks, waves * pairs);      // the first one of the rest
        int shared = task * w.steps;
        if constexpr (FORM == kWeightGrad) {
            const int per = w.tiles * w.tiles_b, e = task / per;
            shared = task == tasks ? before : sh.before[e] + (task - e * per) * steps_of(w, sh.count[e]);
        }
        const int rest = before - shared;
        // every pair takes part where that leaves it kMinPart steps or a tile
        const int parts = min(pairs, max(tasks - task, rest / (widest <= 64 ? kMinPart : kMinPartWide)));
        // with few rows more stages fit the ring: more of the weights are under way
        const int half = FORM == kWeightGrad ? 128 : (widest + 31) / 32 * 16;
        sh.stage_bytes = kABytes + loaded_rows(half) * 128;
        sh.stages = FORM == kWeightGrad ? kStages : min(kMaxStages, kStages * kStageBytes / sh.stage_bytes);
        sh.tasks = tasks;
        sh.waves = waves;
        sh.shared = shared;
        sh.parts = parts;
        sh.base = parts ? rest / parts : 0;
        sh.more = parts ? rest - sh.base * parts : 0;
    }
    if (bad && (int)blockIdx.x == 2 * sh.first_pair) flag_status(p.dev_status, MOE_ERR_INVALID_ARG);
    __syncwarp();
}

__device__ __forceinline__ int arrived(const int32_t *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// ---------------------------------------------------------------- loads

// d_w: rows of the expert in step c, steps of the MMA that they take, and whether rows of
// others are in the last one.
__device__ __forceinline__ int valid_rows(int count, int c) { return min(kStep, count - c * kStep); }
__device__ __forceinline__ int mma_steps(int valid) { return (valid + 15) / 16; }
__device__ __forceinline__ bool ragged_step(const Segment &g, int count, int c)
{
    return c == g.steps - 1 && count % kStep != 0;
}

template <int FORM>
__device__ __forceinline__ void load_steps(Shared &sh, uint8_t *ring, const Args &p, const Maps &maps, const Shape &w)
{
    const uint32_t rank = cluster_rank();
    Walk<FORM> walk(sh, p, w);
    Segment g;
    const int stages = FORM == kWeightGrad ? kStages : sh.stages;
    const int stage_bytes = FORM == kWeightGrad ? kStageBytes : sh.stage_bytes;
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
        if (FORM == kWeightGrad && sh.count[g.e] == 0) continue;
        const int half = g.cols / 2;
        const int a0 = g.tile * kTileRows + rank * 128;      // first row of A
        const int start = sh.start[g.e], count = sh.count[g.e];
        const int b_bytes = FORM == kWeightGrad ? (half > 64 ? 2 : 1) * 8192 : loaded_rows(half) * 128;
        for (int c = g.c0; c < g.c1; c++) {
            if (!(ok = mbar_wait_cluster(&sh.empty[s], phase ^ 1, &sh.dead))) break;
            if (elect_lane()) {
                uint8_t *at = ring + s * stage_bytes, *bt = at + kABytes;
                uint32_t bar = cluster_addr(&sh.full[s], 0);
                if constexpr (FORM == kWeightGrad) {
                    // the last rows of an expert go by this CTA's warp that clears what is behind
                    // them.  (A barrier of the pair that both CTAs arrive at in every step took
                    // twice the time: 242 us for 116.)
                    if (ragged_step(g, count, c)) {
                        bar = smem_addr(&sh.landed[s]);
                        mbar_expect(&sh.landed[s], kABytes + b_bytes);
                        if (rank == 0) mbar_arrive(&sh.full[s]);
                    } else if (rank == 0) {
                        mbar_expect(&sh.full[s], 2 * (kABytes + b_bytes));
                    }
                    const int r = start + c * kStep;
                    tile_load2(at, &maps.a, a0, r, bar);
                    tile_load2(at + 8192, &maps.a, a0 + 64, r, bar);
                    const int b0 = g.row0 + rank * half;
                    tile_load2(bt, &maps.b[0], b0, r, bar);
                    if (half > 64) tile_load2(bt + 8192, &maps.b[0], b0 + 64, r, bar);
                } else {
                    if (rank == 0) mbar_expect(&sh.full[s], 2 * (kABytes + b_bytes));
                    const int l = c * kStep;
                    if constexpr (FORM == kPlain) {
                        tile_load3(at, &maps.a, l, a0, g.e, bar);
                    } else if constexpr (FORM == kGated) {
                        tile_load5(at, &maps.a, l, 0, 0, a0 / 16, g.e, bar);
                    } else {
                        tile_load3(at, &maps.a, a0, l, g.e, bar);
                        tile_load3(at + 8192, &maps.a, a0 + 64, l, g.e, bar);
                    }
                    const int r = start + g.row0 + rank * half;
                    if (half <= 32) {
                        tile_load2(bt, &maps.b[0], l, r, bar);
                        if (half > 16) tile_load2(bt + 2048, &maps.b[0], l, r + 16, bar);
                    } else {
                        tile_load2(bt, half <= 64 ? &maps.b[1] : &maps.b[2], l, r, bar);
                    }
                }
            }
            __syncwarp();
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
    }
    // the stages in use come free before the CTA ends: then no copy, MMA or arrival is under way
    for (int i = 0; ok && i < stages; i++) {
        ok = mbar_wait_cluster(&sh.empty[s], phase ^ 1, &sh.dead);
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!ok) {      // a wait gave up: the copies in flight are given a hundred times what one takes
        const uint64_t now = global_ns();
        while (global_ns() - now < 200000) {}
    }
}

// The stages of d_w that hold the last rows of an expert: the rows behind them, up to the MMA's
// next 16, are cleared in both operands.
__device__ __forceinline__ void clear_steps(Shared &sh, uint8_t *ring, const Args &p, const Shape &w)
{
    const int lane = threadIdx.x & 31;
    Walk<kWeightGrad> walk(sh, p, w);
    Segment g;
    int s = 0;
    uint32_t phases = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
        const int count = sh.count[g.e];
        if (count == 0) continue;
        const int ahead = g.c1 - g.c0;
        if (ragged_step(g, count, g.c1 - 1)) {
            const int last = (s + ahead - 1) % kStages;
            if (!(ok = mbar_wait_warp(&sh.landed[last], phases >> last & 1, &sh.dead))) break;
            phases ^= 1u << last;
            const int valid = valid_rows(count, g.c1 - 1), to = 16 * mma_steps(valid);
            // row r of the operands' four atoms, 128 bytes each
            uint8_t *stage = ring + last * kStageBytes;
            for (int i = lane; i < (to - valid) * 32; i += 32) {
                const int r = valid + (i >> 5), atom = i >> 3 & 3;
                *(int4 *)(stage + atom * 8192 + r * 128 + (i & 7) * 16) = make_int4(0, 0, 0, 0);
            }
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(cluster_addr(&sh.cleared[last], 0));
        }
        s = (s + ahead) % kStages;
    }
}

// ---------------------------------------------------------------- MMA

template <int FORM>
__device__ __forceinline__ void issue_steps(Shared &sh, uint8_t *ring, const Args &p, const Shape &w)
{
    constexpr bool kAByK = FORM == kPlain || FORM == kGated, kBByK = FORM != kWeightGrad;
    Walk<FORM> walk(sh, p, w);
    Segment g;
    const int stages = FORM == kWeightGrad ? kStages : sh.stages;
    const int stage_bytes = FORM == kWeightGrad ? kStageBytes : sh.stage_bytes;
    int s = 0, d = 0;
    uint32_t phase = 0, sums_phase = 0, cleared = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
        if (FORM == kWeightGrad && sh.count[g.e] == 0) continue;
        const uint32_t word = mma_pair_word(g.cols, kAByK, kBByK);
        const int most = FORM == kWeightGrad ? kSumSteps : g.steps;     // steps of a sum in tensor memory
        int left = 0;
        for (int c = g.c0; c < g.c1; c++) {
            const bool fresh = left == 0;
            if (fresh) {
                left = min(most, g.c1 - c);
                if (!(ok = mbar_wait_cluster(&sh.sums_empty[d], sums_phase ^ 1, &sh.dead))) break;
                tmem_fence_after();
            }
            left--;
            const uint32_t sums = sh.tmem + d * kTileRows;
            if (!(ok = mbar_wait_cluster(&sh.full[s], phase, &sh.dead))) break;
            if (FORM == kWeightGrad && ragged_step(g, sh.count[g.e], c)) {
                if (!(ok = mbar_wait_cluster(&sh.cleared[s], cleared >> s & 1, &sh.dead))) break;
                cleared ^= 1u << s;
            }
            tmem_fence_after();
            const uint32_t at = smem_addr(ring) + s * stage_bytes, bt = at + kABytes;
            const uint64_t a = kAByK ? mma_smem_word(at, 1024) : mma_across_word(at, 8192);
            const uint64_t b = kBByK ? mma_smem_word(bt, 1024) : mma_across_word(bt, 8192);
            const int n = FORM == kWeightGrad ? mma_steps(valid_rows(sh.count[g.e], c)) : 4;
            if (elect_lane()) {
#pragma unroll
                for (int i = 0; i < 4; i++)     // 16 of the sum: 32 bytes along it, 2 KiB across
                    if (FORM != kWeightGrad || i < n)
                        mma_bf16_pair(sums, a + (uint64_t)(i * (kAByK ? 2 : 128)),
                                      b + (uint64_t)(i * (kBByK ? 2 : 128)), word, !fresh || i > 0);
                mma_commit_pair(&sh.empty[s]);
                if (left == 0) mma_commit_pair(&sh.sums_full[d]);
            }
            __syncwarp();
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
            if (left == 0) {
                d ^= 1;
                if (d == 0) sums_phase ^= 1;
            }
        }
    }
}

// ---------------------------------------------------------------- the end of a tile

struct Finish {
    int first, parts;          // parts of a cut tile: the pair that has the first one, how many
    int here;                  // which of them this CTA holds
    const float *from;         // this thread's place in the first one
};

// A part's sums: a block of 16 columns is 4 x 128 threads x 4 values, so that a thread moves
// 16 bytes at a time.
__device__ __forceinline__ void store_part(float *part, int c0, const float (&v)[kCols])
{
#pragma unroll
    for (int j = 0; j < kCols; j += 4)
        __stcg((float4 *)(part + (c0 + j) * 128), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
}
__device__ __forceinline__ const float *parts_from(const Shared &sh, const Args &p, const Finish &f)
{
    return p.partial + (int64_t)(4 * (sh.first_pair + f.first) + 2 * cluster_rank()) * kPart + (threadIdx.x & 127) * 4;
}
__device__ __forceinline__ void load_part(const Finish &f, int q, int c0, float (&v)[kCols])
{
    // a part that starts the tile is its pair's last, any other its first
    const float *part = f.from + (4 * q + (q == 0)) * kPart;
#pragma unroll
    for (int j = 0; j < kCols; j += 4) {
        const float4 x = __ldcg((const float4 *)(part + (c0 + j) * 128));
        v[j] = x.x, v[j + 1] = x.y, v[j + 2] = x.z, v[j + 3] = x.w;
    }
}

// The sums of a cut tile in columns c0 .. c0 + 15 over all of its parts in their order; v holds this
// CTA's part.
template <int AHEAD>      // parts whose loads are in flight
__device__ __forceinline__ void add_parts(const Finish &f, int c0, float (&v)[kCols])
{
    float sum[kCols] = {};
    for (int q0 = 0; q0 < f.parts; q0 += AHEAD) {
        float x[AHEAD][kCols];
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            if (q0 + i < f.parts && q0 + i != f.here) load_part(f, q0 + i, c0, x[i]);
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            if (q0 + i < f.parts)
#pragma unroll
                for (int j = 0; j < kCols; j++) sum[j] += q0 + i == f.here ? v[j] : x[i][j];
    }
#pragma unroll
    for (int j = 0; j < kCols; j++) v[j] = sum[j];
}

// The same with all parts in memory.
__device__ __forceinline__ void read_parts(const Finish &f, int c0, float (&v)[kCols])
{
#pragma unroll
    for (int j = 0; j < kCols; j++) v[j] = 0.f;
#pragma unroll 1
    for (int q = 0; q < f.parts; q++) {
        float x[kCols];
        load_part(f, q, c0, x);
#pragma unroll
        for (int j = 0; j < kCols; j++) v[j] += x[j];
    }
}

// Where this segment is part of a cut tile: its parts.
__device__ __forceinline__ void find_parts(const Shared &sh, const Segment &g, Finish &f)
{
    f.parts = 1;
    if (g.c1 - g.c0 == g.steps) return;
    f.first = owner_of(sh, g.unit);
    f.parts = owner_of(sh, g.unit + g.steps - 1) - f.first + 1;
    f.here = (int)(blockIdx.x / 2) - sh.first_pair - f.first;
}

// By all of the CTA's finishing warps: whether they are to finish the tile, which falls to the part that
// is done last (`early`: all others had arrived before).  Any other goes to memory by `store(slot)`.
template <typename Store>
__device__ __forceinline__ bool join_parts(Shared &sh, const Args &p, const Segment &g, Finish &f, bool early, Store store)
{
    if (f.parts == 1 || early) return true;
    // (the thread's place among the 128 of a row block is the same for the warps that share its columns)
    store(p.partial + (int64_t)(2 * blockIdx.x + (g.c0 == 0)) * kPart + (threadIdx.x & 127) * 4);
    __threadfence();
    named_barrier(1, kFinishWarps * 32);
    if (threadIdx.x == 0) sh.last = atomicAdd(p.arrivals + 2 * f.first + cluster_rank(), 1) == f.parts - 1;
    named_barrier(1, kFinishWarps * 32);
    const bool last = sh.last;
    __threadfence();
    return last;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The warp's staging: 16 rows of 64 bytes (32: half of them), whose 16-byte pieces are XOR-ed by
// the row, so that eight rows at one piece, or eight pieces in a row, are on different banks.
template <int PIECES>
__device__ __forceinline__ uint8_t *staged(uint8_t *staging, int row, int piece)
{
    return staging + row * (16 * PIECES) + ((piece ^ (PIECES == 4 ? row >> 1 & 3 : row >> 2 & 1)) << 4);
}

// Rows c0 .. c0 + 15 of a tile in staging to rows `pitch` values apart, the first `rows` of them and
// their first `width` outputs (16 to a row for two pieces, 32 for four).
template <int PIECES>
__device__ __forceinline__ void rows_out(uint8_t *staging, __nv_bfloat16 *to, int64_t pitch, int rows, int width)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kCols * PIECES / 32; i++) {
        const int at = i * 32 + lane, row = at / PIECES, piece = at % PIECES;
        if (row < rows && piece * 8 < width)
            *(int4 *)(to + row * pitch + piece * 8) = *(const int4 *)staged<PIECES>(staging, row, piece);
    }
}

// Values of two rows and one output each, in 8 x 8 matrices (tmem_load_matrices), into staging:
// matrix (h, u) of rows 8 g .. 8 g + 7 is its piece PIECE(h, u).
template <typename Piece>
__device__ __forceinline__ void stage(uint8_t *staging, const float (&v)[kCols], Piece piece)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < 2; g++) {
        uint32_t r[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int i = 8 * (q >> 1) + 4 * g + 2 * (q & 1);
            r[q] = bf16_pair(v[i], v[i + 1]);
        }
        store_matrices(staged<4>(staging, 8 * g + (lane & 7), piece(lane >> 4, lane >> 3 & 1)), r);
    }
}

// Rows c0 .. c0 + 15 of a tile from their sums v.  `first`: the first row, `rows`: how many there
// are, n0: the warp's first output.
template <int FORM>
__device__ __forceinline__ void finish_rows(const Args &p, uint8_t *staging, const float (&v)[kCols], int64_t first,
                                            int rows, int n0, const int4 (&gates)[4])
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if constexpr (FORM == kGated) {
        // lanes 16 h + .. of a matrix (h, 0) have the gates of outputs 8 h + .., of (h, 1) their ups
        uint32_t r[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int i = 8 * (q & 1) + 4 * (q >> 1);
            r[q] = bf16_pair(gated_output(v[i], v[i + 2]), gated_output(v[i + 1], v[i + 3]));
        }
        store_matrices(staged<2>(staging, 8 * (lane >> 4) + (lane & 7), lane >> 3 & 1), r);
        if (p.keep) stage(staging + kCols * 32, v, [](int h, int u) { return 2 * u + h; });
        __syncwarp();
        rows_out<2>(staging, p.out + first * p.N + n0, p.N, rows, p.N - n0);
        if (p.keep) {
            // pieces 0, 1 of a row are of gate, 2, 3 of up
            __nv_bfloat16 *const to = p.keep + first * 2 * p.N + n0;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int at = i * 32 + lane, row = at / 4, piece = at % 4;
                if (row < rows && n0 + (piece & 1) * 8 < p.N)
                    *(int4 *)(to + (int64_t)row * 2 * p.N + (piece >> 1) * p.N + (piece & 1) * 8) =
                        *(const int4 *)staged<4>(staging + kCols * 32, row, piece);
            }
        }
    } else if constexpr (FORM == kGateGrad) {
        const int K = p.K;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int at = (i & 1) * 32 + lane;
            *(int4 *)staged<4>(staging + (i >> 1) * kCols * 64, at / 4, at % 4) = gates[i];
        }
        __syncwarp();
        float d_gate[kCols], d_up[kCols];
#pragma unroll
        for (int g = 0; g < 2; g++) {
            uint32_t gate[4], up[4];
            uint8_t *const at = staged<4>(staging, 8 * g + (lane & 7), lane >> 3);
            load_matrices(at, gate);
            load_matrices(at + kCols * 64, up);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int i = 8 * (q >> 1) + 4 * g + 2 * (q & 1);
                gated_gradient(__uint_as_float(gate[q] << 16), __uint_as_float(up[q] << 16), v[i], d_gate[i], d_up[i]);
                gated_gradient(__uint_as_float(gate[q] & 0xffff0000u), __uint_as_float(up[q] & 0xffff0000u), v[i + 1],
                               d_gate[i + 1], d_up[i + 1]);
            }
        }
        __syncwarp();
        stage(staging, d_gate, [](int h, int u) { return 2 * h + u; });
        stage(staging + kCols * 64, d_up, [](int h, int u) { return 2 * h + u; });
        __syncwarp();
        rows_out<4>(staging, p.out + first * 2 * K + n0, 2 * K, rows, K - n0);
        rows_out<4>(staging + kCols * 64, p.out + first * 2 * K + K + n0, 2 * K, rows, K - n0);
    } else {
        stage(staging, v, [](int h, int u) { return 2 * h + u; });
        __syncwarp();
        rows_out<4>(staging, p.out + first * p.rows_a + n0, p.rows_a, rows, p.rows_a - n0);
    }
}

// Gate and up of 16 rows for the warp's 32 outputs, as they go into the staging.
__device__ __forceinline__ void load_gates(const Args &p, int64_t first, int rows, int n0, int4 (&gates)[4])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int at = (i & 1) * 32 + lane, row = at / 4, piece = at % 4;
        gates[i] = make_int4(0, 0, 0, 0);
        if (row < rows && n0 + piece * 8 < p.K)
            gates[i] = ld_stream((const int4 *)(p.pre + (first + row) * 2 * p.K + (i >> 1) * p.K + n0 + piece * 8));
    }
}

// d_w: 64 bytes of each of the warp's 32 rows, the first at (e, n0, k), by one tile store, which writes
// what is inside the matrix.
__device__ __forceinline__ void weights_out(const CUtensorMap *map, uint8_t *staging, const uint32_t (&words)[16], int e,
                                            int n0, int k)
{
    const int lane = threadIdx.x & 31;
    if (lane == 0) tile_stores_read();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; i++)
        *(uint4 *)staged<4>(staging, lane, i) = make_uint4(words[4 * i], words[4 * i + 1], words[4 * i + 2], words[4 * i + 3]);
    async_proxy_fence();
    __syncwarp();
    if (lane == 0) tile_store3(map, k, n0, e, staging);
}

// The other parts of a cut tile into the ring, when it is no longer in use: all of their loads at once, where
// they fit (82 rows over 2 experts of 2,496 x 3,808: 17.8 us, 19 a block of columns at a time).  A thread
// reads what it has copied itself.
constexpr int kRingBlocks = kStages * kStageBytes / (kFinishWarps * 32 * kCols * 4);
__device__ __forceinline__ int4 *ring_block(uint8_t *ring, int i, int j)
{
    return (int4 *)ring + (i * (kCols / 4) + j) * (kFinishWarps * 32) + threadIdx.x;
}
__device__ __forceinline__ void copy_parts(uint8_t *ring, const Finish &f, int c0, int turn, int rows)
{
    int i = 0;
    for (int q = 0; q < f.parts; q++) {
        if (q == f.here) continue;
        const float *part = f.from + (4 * q + (q == 0)) * kPart;
        for (int c = c0; c < rows; c += turn, i++)
#pragma unroll
            for (int j = 0; j < kCols / 4; j++)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(ring_block(ring, i, j))),
                             "l"(part + (c + 4 * j) * 128)
                             : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}
// Block b (of `blocks`) of the tile out of them, over all parts in their order.
__device__ __forceinline__ void add_copies(uint8_t *ring, const Finish &f, int b, int blocks, float (&v)[kCols])
{
    float sum[kCols] = {};
    for (int q = 0, i = b; q < f.parts; q++) {
        if (q == f.here) {
#pragma unroll
            for (int j = 0; j < kCols; j++) sum[j] += v[j];
            continue;
        }
#pragma unroll
        for (int j = 0; j < kCols / 4; j++) {
            const float4 x = *(const float4 *)ring_block(ring, i, j);
            sum[4 * j] += x.x, sum[4 * j + 1] += x.y, sum[4 * j + 2] += x.z, sum[4 * j + 3] += x.w;
        }
        i += blocks;
    }
#pragma unroll
    for (int j = 0; j < kCols; j++) v[j] = sum[j];
}

template <int FORM>
__device__ __forceinline__ void finish_steps(Shared &sh, uint8_t *ring, uint8_t *staging, const Args &p, const Shape &w)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3, group = warp >> 2;
    constexpr int kTurn = kGroups * kCols;
    const uint32_t rank = cluster_rank();
    staging += warp * kStaging;
    Walk<FORM> walk(sh, p, w);
    Segment g;
    int d = 0;
    uint32_t phase = 0;
    while (walk.next(g)) {
        const int a_row = g.tile * kTileRows + rank * 128 + quarter * 32;    // the warp's first row of A
        const int64_t first = sh.start[g.e] + g.row0;
        int4 gates[4];                                   // loaded a block of rows ahead
        if constexpr (FORM == kGateGrad) load_gates(p, first + group * kCols, g.rows - group * kCols, a_row, gates);
        Finish f;
        find_parts(sh, g, f);
        const bool others = f.parts > 1 && arrived(p.arrivals + 2 * f.first + rank) == f.parts - 1;
        const bool ok = mbar_wait_cluster(&sh.sums_full[d], phase, &sh.dead);
        if (!named_all(1, kFinishWarps * 32, ok)) break;
        const bool early = f.parts > 1 && named_all(1, kFinishWarps * 32, others);
        tmem_fence_after();
        const uint32_t sums = sh.tmem + ((uint32_t)(quarter * 32) << 16) + d * kTileRows;
        const bool finish = join_parts(sh, p, g, f, early, [&](float *slot) {
            for (int c0 = group * kCols; c0 < g.rows; c0 += kTurn) {
                float v[kCols];
                tmem_load_matrices(sums + c0, v);
                store_part(slot, c0, v);
            }
        });
        if (finish) {
            f.from = parts_from(sh, p, f);
            const int blocks = max(0, (g.rows - group * kCols + kTurn - 1) / kTurn);
            // (gate and up in their registers' place: 16,384 rows' gradients take 144 us without, 148 with)
            const bool copied = FORM != kGateGrad && f.parts > 1 && walk.over() && (f.parts - 1) * blocks <= kRingBlocks;
            if (copied) copy_parts(ring, f, group * kCols, kTurn, g.rows);
            int b = 0;
#pragma unroll 1
            for (int c0 = group * kCols; c0 < g.rows; c0 += kTurn, b++) {
                float v[kCols];
                int4 next[4];
                if constexpr (FORM == kGateGrad) load_gates(p, first + c0 + kTurn, g.rows - c0 - kTurn, a_row, next);
                tmem_load_matrices(sums + c0, v);
                if (copied) add_copies(ring, f, b, blocks, v);
                else if (f.parts > 1) add_parts<FORM == kGateGrad ? 1 : 4>(f, c0, v);
                finish_rows<FORM>(p, staging, v, first + c0, g.rows - c0, FORM == kGated ? a_row / 2 : a_row, gates);
                if constexpr (FORM == kGateGrad)
#pragma unroll
                    for (int i = 0; i < 4; i++) gates[i] = next[i];
            }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(cluster_addr(&sh.sums_empty[d], 0));
        d ^= 1;
        if (d == 0) phase ^= 1;
    }
}

// d_w.  The tensor core cuts its sums off where they leave fp32, which grows with their length (2,048
// rows: 2.1e-6 of the result, towards zero).  So it sums kSumSteps steps at a time, and these
// warps add them up, rounding to nearest, in registers: a thread has half of the columns of a row
// of D.  (8 experts' 16,384 rows of 2,048 x 1,408 in fp32: 8.4e-7 and 75 us with 12 steps, 5.8e-7 and 84 us
// with 8, 1.1e-6 and 71 us with 16.)  That also hands tensor memory back before the tile is written.
constexpr int kBlocks = kTileRows / kCols / kGroups;

__device__ __forceinline__ void finish_weights(Shared &sh, uint8_t *staging, const Args &p, const Maps &maps, const Shape &w)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3, group = warp >> 2;
    const uint32_t rank = cluster_rank();
    staging += warp * kStaging;
    Walk<kWeightGrad> walk(sh, p, w);
    Segment g;
    int d = 0;
    uint32_t phase = 0;
    // block b of this warp: 32 columns by the groups in turn
    auto column = [&](int b) { return ((b >> 1) * kGroups + group) * 32 + (b & 1) * kCols; };
    while (walk.next(g)) {
        float sum[kBlocks][kCols] = {};
        bool ok = true;
        const int to = g.c1, cols = g.cols;
        for (int c = sh.count[g.e] ? g.c0 : to; ok && c < to; c += kSumSteps) {
            if (!(ok = mbar_wait_cluster(&sh.sums_full[d], phase, &sh.dead))) break;
            tmem_fence_after();
            const uint32_t sums = sh.tmem + ((uint32_t)(quarter * 32) << 16) + d * kTileRows;
#pragma unroll
            for (int b = 0; b < kBlocks; b++)
                if (column(b) < cols) {
                    float v[kCols];
                    tmem_load(sums + column(b), v);
#pragma unroll
                    for (int j = 0; j < kCols; j++) sum[b][j] += v[j];
                }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(cluster_addr(&sh.sums_empty[d], 0));
            d ^= 1;
            if (d == 0) phase ^= 1;
        }
        if (!named_all(1, kFinishWarps * 32, ok)) break;
        const int a_row = g.tile * kTileRows + rank * 128 + quarter * 32;    // the warp's first row of A
        Finish f;
        find_parts(sh, g, f);
        // (the last one reads all parts from memory: what it holds has no registers beside them)
        const bool finish = join_parts(sh, p, g, f, false, [&](float *slot) {
#pragma unroll
            for (int b = 0; b < kBlocks; b++)
                if (column(b) < g.cols) store_part(slot, column(b), sum[b]);
        });
        if (!finish || a_row >= p.N) continue;
        if (f.parts > 1) f.from = parts_from(sh, p, f);
#pragma unroll
        for (int b = 0; b < kBlocks; b += 2) {
            if (column(b) >= g.rows) break;
            if (f.parts > 1)
#pragma unroll
                for (int i = 0; i < 2; i++) read_parts(f, column(b + i), sum[b + i]);
            uint32_t words[16];
            if (p.d_w_f32) {
#pragma unroll
                for (int i = 0; i < 2; i++)
                    if (column(b + i) < g.rows) {
#pragma unroll
                        for (int j = 0; j < kCols; j++) words[j] = __float_as_uint(sum[b + i][j]);
                        weights_out(&maps.d, staging, words, g.e, a_row, g.row0 + column(b + i));
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 16; j++) words[j] = bf16_pair(sum[b + j / 8][j % 8 * 2], sum[b + j / 8][j % 8 * 2 + 1]);
                weights_out(&maps.d, staging, words, g.e, a_row, g.row0 + column(b));
            }
        }
    }
    if (lane == 0) tile_stores_done();
}

// The places in shared memory that do not depend on the product.
struct Memory {
    uint8_t *ring;
    Shared &sh;
    __device__ Memory(uint8_t *raw)
        : ring(raw + (1024 - (smem_addr(raw) & 1023)) % 1024),
          sh(*(Shared *)(ring + kStages * kStageBytes + kFinishWarps * kStaging))
    {
    }
};

// Before the work is known: barriers, tensor memory, tensor maps, the pair's other CTA, and then the wait
// for the kernel before, whose end all that runs beside.
__device__ __forceinline__ void start(Shared &sh, int warp, const Maps &maps, const Maps &maps_w)
{
    const int lane = threadIdx.x & 31;
    if (warp == kWarpLoad) {
        if (lane == 0) {
            map_prefetch(&maps.a);
            map_prefetch(&maps.b[0]);
            if (&maps != &maps_w) {
                map_prefetch(&maps_w.a);
                map_prefetch(&maps_w.b[0]);
            }
            sh.dead = 0;
            sh.first_pair = 0;
            sh.pairs = gridDim.x / 2;
        }
    } else if (warp == kWarpMma) {
        if (lane < kMaxStages) {
            mbar_init(&sh.full[lane], 1);
            mbar_init(&sh.empty[lane], 1);
        }
        if (lane < kStages) {
            mbar_init(&sh.landed[lane], 1);
            mbar_init(&sh.cleared[lane], 2);
        }
        if (lane < 2) {
            mbar_init(&sh.sums_full[lane], 1);
            mbar_init(&sh.sums_empty[lane], 2 * kFinishWarps);
        }
        mbar_init_fence();
    } else if (warp == kWarpClear) {
        tmem_alloc_pair(&sh.tmem, kTmemColumns);
        tmem_fence_before();
    }
    cluster_barrier();
    tmem_fence_after();
    pdl_wait();
    pdl_trigger();
}

// By all threads, after the load warp's scan.
template <int FORM>
__device__ __forceinline__ void run_product(uint8_t *ring, Shared &sh, int warp, const Maps &maps, const Args &p)
{
    const Shape shape = shape_of<FORM>(p);
    uint8_t *staging = ring + kStages * kStageBytes;
    if (warp == kWarpLoad) {
        load_steps<FORM>(sh, ring, p, maps, shape);
    } else if (warp == kWarpMma) {
        if (cluster_rank() == 0) issue_steps<FORM>(sh, ring, p, shape);
    } else if (warp == kWarpClear) {
        if constexpr (FORM == kWeightGrad) clear_steps(sh, ring, p, shape);
    } else {
        if constexpr (FORM == kWeightGrad) finish_weights(sh, staging, p, maps, shape);
        else finish_steps<FORM>(sh, ring, staging, p, shape);
    }
}

__device__ __forceinline__ void end(Shared &sh, int warp, uint32_t *dev_status)
{
    tmem_fence_before();
    __syncthreads();
    cluster_barrier();
    if (warp == kWarpClear) {
        if (sh.dead && (threadIdx.x & 31) == 0) flag_status(dev_status, MOE_ERR_TIMEOUT);
        tmem_fence_after();
        tmem_free_pair(sh.tmem, kTmemColumns);
    }
}

template <int FORM>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_expert_product(const __grid_constant__ Maps maps, const __grid_constant__ Args p)
{
    extern __shared__ uint8_t raw[];
    const Memory m(raw);
    const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
    start(m.sh, warp, maps, maps);
    if (warp == kWarpLoad) scan_experts<FORM>(m.sh, p, shape_of<FORM>(p));
    __syncthreads();
    run_product<FORM>(m.ring, m.sh, warp, maps, p);
    end(m.sh, warp, p.dev_status);
}

// Pairs for the rows' gradient where both gradients are taken at once, by what they take: their steps,
// and those that the end of a tile is worth by what it reads and writes.  By one warp, the same in
// every CTA.  (Counting the turns of each side for every split took longer than it won.)
__device__ __forceinline__ int split_pairs(const Args &p, const Args &p_w)
{
    const int rows_end = p.pre ? 8 : 6, weights_end = p.d_w_f32 ? 8 : 6;
    const Shape a = shape_of<kRowGrad>(p), w = shape_of<kWeightGrad>(p_w);
    int tiles = 0, steps = 0;
    bool bad = false;
    for (int e = threadIdx.x & 31; e < p.E; e += 32) {
        int start, count;
        expert_rows(p.offsets, p.counts, p.block_rows, p.a_rows, e, start, count, bad);
        tiles += row_tiles(count, p.most);
        steps += steps_of(w, count) + weights_end;
    }
    const float rows = (float)__reduce_add_sync(kFull, tiles) * (float)(a.tiles * (a.steps + rows_end));
    const float weights = (float)__reduce_add_sync(kFull, steps) * (float)(w.tiles * w.tiles_b);
    const int pairs = gridDim.x / 2;
    return rows == 0.f ? 0 : min(pairs - 1, max(1, (int)((float)pairs * rows / (rows + weights) + 0.5f)));
}

// Both gradients in one launch, each on pairs of its own: one start and one end, and one's stores beside
// the other's MMAs (8 experts' 4,096 rows of 2,048 x 1,408: 63 us, 71 in two launches; 300 rows of 328 x 648
// in five experts: 13 us, 19, before smaller tiles made it 11).
template <int FORM>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_expert_gradients(const __grid_constant__ Maps maps, const __grid_constant__ Args p,
                       const __grid_constant__ Maps maps_w, const __grid_constant__ Args p_w)
{
    extern __shared__ uint8_t raw[];
    const Memory m(raw);
    const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
    start(m.sh, warp, maps, maps_w);
    if (warp == kWarpLoad) {
        const int split = split_pairs(p, p_w);
        const bool weights = (int)blockIdx.x / 2 >= split;
        if ((threadIdx.x & 31) == 0) {
            m.sh.first_pair = weights ? split : 0;
            m.sh.pairs = weights ? gridDim.x / 2 - split : split;
            m.sh.weights = weights;
        }
        __syncwarp();
        if (weights) scan_experts<kWeightGrad>(m.sh, p_w, shape_of<kWeightGrad>(p_w));
        else scan_experts<FORM>(m.sh, p, shape_of<FORM>(p));
    }
    __syncthreads();
    if (m.sh.weights) run_product<kWeightGrad>(m.ring, m.sh, warp, maps_w, p_w);
    else run_product<FORM>(m.ring, m.sh, warp, maps, p);
    end(m.sh, warp, p.dev_status);
}

// Clears the arrival counters of cut tiles.
__global__ void __launch_bounds__(2 * kMaxCtas) k_product_begin(int32_t *arrivals)
{
    pdl_trigger();
    pdl_wait();
    arrivals[threadIdx.x] = 0;
}

// ---------------------------------------------------------------- launch

// A tensor map of bf16 or fp32 values: `dims` sizes, strides in values from the second dimension on.
struct MapSpec {
    const void *base;
    int dims;
    uint64_t size[5], stride[4];
    uint32_t box[5];
    bool f32 = false;
};
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn *out)
{
    static EncodeFn known = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got) !=
                cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return (EncodeFn)fn;
    }();
    *out = known;
    return known ? cudaSuccess : cudaErrorNotSupported;
}

cudaError_t encode(CUtensorMap *map, const MapSpec &m)
{
    EncodeFn fn;
    const cudaError_t err = encode_fn(&fn);
    if (err != cudaSuccess) return err;
    cuuint64_t strides[4];
    cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i + 1 < m.dims; i++) strides[i] = m.stride[i] * (m.f32 ? 4 : 2);
    const bool bytes64 = m.box[0] * (m.f32 ? 4 : 2) == 64;
    return fn(map, m.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)m.dims,
              const_cast<void *>(m.base), m.size, strides, m.box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// [rows][width] in boxes of 64 columns.
MapSpec rows_map(const void *base, int64_t rows, int64_t width, uint32_t box_rows)
{
    return {base, 2, {(uint64_t)width, (uint64_t)rows}, {(uint64_t)width}, {64, box_rows}};
}
// [E][N][K] weights in boxes of 64 columns.
MapSpec weights_map(const void *base, int64_t E, int64_t N, int64_t K, uint32_t box_rows)
{
    return {base, 3, {(uint64_t)K, (uint64_t)N, (uint64_t)E}, {(uint64_t)K, (uint64_t)(N * K)}, {64, box_rows, 1}};
}
// [E][gate, up][N][K] weights as (K, 8 rows, gate or up, groups of 8 rows, E): a box is 8 groups
// of 8 gate rows and their 8 up rows.
MapSpec gated_map(const void *base, int64_t E, int64_t N, int64_t K)
{
    return {base,
            5,
            {(uint64_t)K, 8, 2, (uint64_t)(N / 8), (uint64_t)E},
            {(uint64_t)K, (uint64_t)(N * K), (uint64_t)(8 * K), (uint64_t)(2 * N * K)},
            {64, 8, 2, 8, 1}};
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
constexpr size_t kPartialBytes = (size_t)2 * kMaxCtas * kPart * 4;

cudaError_t begin(void *ws, cudaStream_t st)
{
    cudaError_t err;
    MOE_TRACED_LAUNCH("k_product_begin", st,
        err = launch_pdl(k_product_begin, dim3(1), dim3(2 * kMaxCtas), 0, st,
                         (int32_t *)((uint8_t *)ws + kPartialBytes)));
    return err;
}

// CTAs of a launch: one per SM, in pairs.
cudaError_t grid_of(int *ctas)
{
    DeviceInfo di;
    const cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    if ((size_t)di.max_smem_optin < kSmem) return cudaErrorInvalidConfiguration;
    *ctas = (di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas) / 2 * 2;
    return cudaSuccess;
}

// Rows of a tile of the B side: half, or a quarter, of 256 where the tiles are few for the pairs all the
// same (2,571 rows of 376 x 1,856: 16.5 us with 256, 12.4 with 128).
int tile_rows(int pairs, int64_t tiles_a, int64_t rows, int64_t experts)
{
    int most = kTileRows;
    while (most > 64 && tiles_a * (2 * rows / most + experts) <= pairs) most /= 2;
    return most;
}

// The shared memory of a kernel, allowed once per device (a bit of `done` each).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (err == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

template <int FORM>
cudaError_t product(const Maps &maps, Args p, int ctas, void *ws, cudaStream_t st)
{
    p.partial = (float *)ws;
    p.arrivals = (int32_t *)((uint8_t *)ws + kPartialBytes);
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(k_expert_product<FORM>, allowed);
    if (err != cudaSuccess) return err;
    MOE_TRACED_LAUNCH("k_expert_product", st,
        err = launch_pdl_cluster(k_expert_product<FORM>, dim3(ctas), dim3(kMmThreads), kSmem, 2, st, maps, p));
    return err;
}

template <int FORM>
cudaError_t gradients(const Maps &maps, Args p, const Maps &maps_w, Args p_w, int ctas, void *ws, cudaStream_t st)
{
    p.partial = p_w.partial = (float *)ws;
    p.arrivals = (int32_t *)((uint8_t *)ws + kPartialBytes);
    p_w.arrivals = p.arrivals + kMaxCtas;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(k_expert_gradients<FORM>, allowed);
    if (err != cudaSuccess) return err;
    MOE_TRACED_LAUNCH("k_expert_gradients", st,
        err = launch_pdl_cluster(k_expert_gradients<FORM>, dim3(ctas), dim3(kMmThreads), kSmem, 2, st, maps, p, maps_w, p_w));
    return err;
}

// Whether tiles of a sum of this length may be cut (scan_experts), so that the counters are needed.
bool may_cut(int sums) { return (sums + kStep - 1) / kStep > kCutSteps; }

// The maps of the rows in boxes of 16, 64 and 128, those that tiles of at most `most` rows use.
cudaError_t row_boxes(Maps &maps, const void *rows, int64_t a_rows, int64_t width, int most)
{
    const uint32_t box[3] = {16, 64, 128};
    const int64_t half = (a_rows < most ? (a_rows + 31) / 32 * 32 : most) / 2;
    cudaError_t err = encode(&maps.b[0], rows_map(rows, a_rows, width, box[0]));
    for (int i = 1; i < 3 && err == cudaSuccess && half > box[i] / 2; i++)
        err = encode(&maps.b[i], rows_map(rows, a_rows, width, box[i]));
    return err;
}

}  // namespace

size_t expert_product_ws_bytes() { return kPartialBytes + align256(2 * kMaxCtas * 4); }

cudaError_t launch_expert_product(const uint16_t *a, int a_rows, const int32_t *offsets,
                                  const int32_t *counts, int block_rows, const uint16_t *w, int E,
                                  int N, int K, bool gated, uint16_t *y, uint16_t *pre, void *ws,
                                  uint32_t *dev_status, cudaStream_t st)
{
    if (a_rows == 0) return cudaSuccess;
    int ctas;
    cudaError_t err = grid_of(&ctas);
    if (err != cudaSuccess) return err;
    const int rows_w = gated ? 2 * N : N;
    const int most = tile_rows(ctas / 2, (rows_w + kTileRows - 1) / kTileRows, a_rows, a_rows < E ? a_rows : E);
    Maps maps = {};
    err = encode(&maps.a, gated ? gated_map(w, E, N, K) : weights_map(w, E, N, K, 128));
    if (err == cudaSuccess) err = row_boxes(maps, a, a_rows, K, most);
    if (err != cudaSuccess) return err;
    const Args p{offsets, counts, block_rows, a_rows, E, N, K, rows_w, K, most, (__nv_bfloat16 *)y,
                 (__nv_bfloat16 *)pre, nullptr, false, nullptr, nullptr, dev_status};
    if (may_cut(K)) err = begin(ws, st);
    if (err != cudaSuccess) return err;
    return gated ? product<kGated>(maps, p, ctas, ws, st) : product<kPlain>(maps, p, ctas, ws, st);
}

cudaError_t launch_expert_product_backward(const uint16_t *d_y, const uint16_t *a, int a_rows,
                                           const int32_t *offsets, const int32_t *counts,
                                           int block_rows, const uint16_t *w, const uint16_t *pre,
                                           int E, int N, int K, uint16_t *d_a, void *d_w,
                                           int d_w_type, void *ws, uint32_t *dev_status,
                                           cudaStream_t st)
{
    if (a_rows == 0)        // no rows: the weights' gradient is zero
        return d_w ? cudaMemsetAsync(d_w, 0, (size_t)E * N * K * (d_w_type == MOE_TYPE_F32 ? 4 : 2), st)
                   : cudaSuccess;
    int ctas;
    cudaError_t err = grid_of(&ctas);
    if (err != cudaSuccess) return err;
    const int pairs = d_a && d_w ? ctas / 4 : ctas / 2;
    const int64_t tiles_n = (N + kTileRows - 1) / kTileRows, tiles_k = (K + kTileRows - 1) / kTileRows;
    Args p{offsets, counts, block_rows, a_rows, E, N, K, K, N, tile_rows(pairs, tiles_k, a_rows, a_rows < E ? a_rows : E),
           (__nv_bfloat16 *)d_a, nullptr, (const __nv_bfloat16 *)pre, d_w_type == MOE_TYPE_F32, nullptr, nullptr,
           dev_status};
    Args p_w = p;
    p_w.most = tile_rows(pairs, E * tiles_n, K, 1);
    Maps maps = {}, maps_w = {};
    if (d_a) {
        err = encode(&maps.a, weights_map(w, E, N, K, 64));
        if (err == cudaSuccess) err = row_boxes(maps, d_y, a_rows, N, p.most);
    }
    if (err == cudaSuccess && d_w) {
        err = encode(&maps_w.a, rows_map(d_y, a_rows, N, 64));
        if (err == cudaSuccess) err = encode(&maps_w.b[0], rows_map(a, a_rows, K, 64));
        MapSpec d = weights_map(d_w, E, N, K, 32);          // boxes of 64 bytes
        d.f32 = p.d_w_f32;
        d.box[0] = p.d_w_f32 ? 16 : 32;
        if (err == cudaSuccess) err = encode(&maps_w.d, d);
    }
    if (err != cudaSuccess) return err;
    if ((d_a && may_cut(N)) || (d_w && may_cut(a_rows))) err = begin(ws, st);
    if (err != cudaSuccess) return err;
    if (d_a && d_w)
        return pre ? gradients<kGateGrad>(maps, p, maps_w, p_w, ctas, ws, st)
                   : gradients<kRowGrad>(maps, p, maps_w, p_w, ctas, ws, st);
    if (d_w) return product<kWeightGrad>(maps_w, p_w, ctas, ws, st);
    if (!d_a) return cudaSuccess;
    return pre ? product<kGateGrad>(maps, p, ctas, ws, st) : product<kRowGrad>(maps, p, ctas, ws, st);
}

}  // namespace moe
