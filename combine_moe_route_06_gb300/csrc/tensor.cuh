// tensor.cuh -- device wrappers of the tensor-core, tensor-memory, bulk-copy
// and mbarrier instructions that the experts' products use.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// ---- mbarriers

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count)
                 : "memory");
}
__device__ __forceinline__ void mbar_init_fence()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Waits until the barrier's phase `parity` is over.  Every wait ends: after
// kWaitLimitNs, or when another thread of the CTA has given up (*dead), the wait
// returns false and *dead is set.
constexpr uint64_t kWaitLimitNs = 5000000000ull;
__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *dead)
{
    if (mbar_try(bar, parity)) return true;
    const uint64_t start = global_ns();
    for (;;) {
        for (int i = 0; i < 64; i++)
            if (mbar_try(bar, parity)) return true;
        if (*dead) return false;
        if (global_ns() - start > kWaitLimitNs) {
            *dead = 1;
            return false;
        }
    }
}

// The same by a whole warp, with one answer for all of its lanes.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *dead)
{
    return __all_sync(kFull, mbar_wait(bar, parity, dead));
}

// Three barriers at once, by a whole warp that polls (a wait on each in turn would
// cost their latencies one after the other, about 100 clocks each).
__device__ __forceinline__ bool mbar_wait3_warp(uint64_t *bar0, uint32_t parity0, uint64_t *bar1,
                                                uint32_t parity1, uint64_t *bar2, uint32_t parity2,
                                                volatile int *dead)
{
    uint64_t start = 0;
    for (int i = 1;; i++) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p, q, r;\n\t"
                     "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
                     "mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
                     "and.pred p, p, q;\n\tand.pred p, p, r;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_addr(bar0)), "r"(parity0), "r"(smem_addr(bar1)), "r"(parity1),
                       "r"(smem_addr(bar2)), "r"(parity2)
                     : "memory");
        if (__all_sync(kFull, ok)) return true;
        if ((i & 63) == 0) {
            const uint64_t now = global_ns();
            if (start == 0) start = now;
            const bool late = now - start > kWaitLimitNs;
            if (late) *dead = 1;
            if (__any_sync(kFull, late || *dead)) return false;
        }
    }
}

// Bytes (a multiple of 16, both ends 16-byte aligned) from global to shared
// memory; the barrier counts them.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// ---- tensor memory: 128 lanes x 512 columns of 32 bits; an address has the
// lane in its upper and the column in its lower 16 bits.

__device__ __forceinline__ void tmem_alloc(uint32_t *out, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(out)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
// 8 or 16 columns of the warp's 32 lanes, ready for use.
template <int COLS>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[COLS])
{
    if constexpr (COLS == 16) {
        uint32_t r[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
              "=r"(r[14]), "=r"(r[15])
            : "r"(addr)
            : "memory");
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
    } else {
        static_assert(COLS == 8, "8 or 16 columns");
        uint32_t r[8];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7])
            : "r"(addr)
            : "memory");
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r[i]);
    }
}

// ---- tcgen05.mma, fp16 operands, fp32 sums: D[128][n] (+)= A[128][16] B[n][16]^T
// with A in tensor memory (a column = two consecutive k) and B in shared memory.

// Instruction word: fp32 D, fp16 A and B, both K-major, n columns, 128 rows.
__device__ __forceinline__ uint32_t mma_f16_word(int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// Shared-memory operand of 8-row groups, each row 64 fp16 (128 bytes) with its
// 16-byte pieces XOR-ed by the row (128-byte swizzle); `group_bytes` apart.
__device__ __forceinline__ uint64_t mma_smem_word(uint32_t addr, uint32_t group_bytes)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
           ((uint64_t)(group_bytes >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t word, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(word), "r"((uint32_t)add)
                 : "memory");
}
// The barrier gets one arrival when all MMAs this thread has issued are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar))
                 : "memory");
}

// One lane of a converged warp, the same for all calls; the compiler keeps what
// the chosen lane issues in uniform registers.
__device__ __forceinline__ bool elect_lane()
{
    uint32_t chosen;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(chosen));
    return chosen != 0;
}

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Barrier `id` of `threads` threads; whether all of them brought true.
__device__ __forceinline__ bool named_all(int id, int threads, bool mine)
{
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all)
                 : "r"(id), "r"(threads), "r"((uint32_t)mine)
                 : "memory");
    return all != 0;
}

// 16 columns of the warp's 32 lanes, as 8 x 8 matrices: v[8 h + 4 g + 2 u + i] is of lane
// 16 h + 8 u + l / 4 and column 8 g + 2 (l % 4) + i, for lane l of the warp.
__device__ __forceinline__ void tmem_load_matrices(uint32_t addr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr), "r"(addr + (16u << 16))
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 matrices of 16-bit values between registers (lane l: row l / 4, columns 2 (l % 4) and
// the next) and shared memory, where they are transposed: lane l gives the address of column l % 8
// of matrix l / 8, 16 bytes.
__device__ __forceinline__ void store_matrices(void *at, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr(at)),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void load_matrices(const void *at, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_addr(at))
                 : "memory");
}

// ---- pairs of CTAs (a cluster of two): the one of rank 0 leads

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster.
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address, in the shared memory of the cluster, of the CTA `rank`'s object that here is at `p`.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_try and mbar_wait_warp for a barrier that the other CTA arrives at too.
__device__ __forceinline__ bool mbar_try_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, volatile int *dead)
{
    bool ok = mbar_try_cluster(bar, parity);
    if (!ok) {
        const uint64_t start = global_ns();
        while (!ok) {
            for (int i = 0; i < 64 && !ok; i++) ok = mbar_try_cluster(bar, parity);
            if (ok || *dead) break;
            if (global_ns() - start > kWaitLimitNs) *dead = 1;
        }
    }
    return __all_sync(kFull, ok);
}

// A tile of a tensor map into this CTA's shared memory; the barrier, here or in the other
// CTA of the pair, counts its bytes.
__device__ __forceinline__ void tile_load2(void *dst, const void *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tile_load3(void *dst, const void *map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tile_load5(void *dst, const void *map, int x, int y, int z, int u, int v, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v)
                 : "memory");
}
// A tile of this CTA's shared memory to a tensor map's place, as one group of this thread; and the
// wait until its groups have been read.
__device__ __forceinline__ void tile_store3(const void *map, int x, int y, int z, const void *src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(map),
                 "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tile_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tile_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void map_prefetch(const void *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// What this thread wrote to shared memory becomes visible to copies and MMAs.
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Both CTAs of a pair call these.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *out, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(out)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

// ---- tcgen05.mma of a pair, bf16 operands in shared memory, fp32 sums:
// D[256][n] (+)= A[256][16] B[n][16]^T.  Each CTA holds 128 rows of A and D and n / 2 rows of B.

// Instruction word; *_by_k: a row's consecutive values are along k, else consecutive rows are
// next to each other in memory.
__host__ __device__ __forceinline__ uint32_t mma_pair_word(int n, bool a_by_k, bool b_by_k)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)!a_by_k << 15) | ((uint32_t)!b_by_k << 16) |
           ((uint32_t)(n >> 3) << 17) | (16u << 24);
}
// Operand along k: 8-row groups 1 KiB apart (mma_smem_word(addr, 1024)).  Operand across k: atoms
// of 64 rows (128 bytes, 16-byte pieces XOR-ed by k % 8) times any number of k, a k 128 bytes
// after the other; `atom_bytes` from an atom to the next 64 rows'.
__device__ __forceinline__ uint64_t mma_across_word(uint32_t addr, uint32_t atom_bytes)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(atom_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t word, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(word), "r"((uint32_t)add)
                 : "memory");
}
// mma_commit at this barrier's place in both CTAs.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
                 "[%0], %1;" ::"r"(smem_addr(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

}  // namespace moe
