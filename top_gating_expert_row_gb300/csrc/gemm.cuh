// Building blocks of the tensor-core kernels (experts' products, adapter
// projection): tensor copies, tcgen05 products with accumulators in tensor
// memory, and the bounded waits that tie a CTA's roles together.
//
// All of them compute D[row][token] = sum_k A[row][k] * B[token][k] with bf16
// operands and fp32 sums: the WEIGHTS are the 128-row operand and the tokens
// the N-wide one (16 to 256 columns), so that one token costs a 16-column
// product instead of a 128-row one, and a CTA's time goes into streaming
// weights, which is what bounds these operators at few tokens.
//
// A k-step is 64 bf16 = one 128-byte swizzled row; a stage of the ring holds 128
// weight rows and the tokens of one k-step. Fewer rows a CTA would not make a
// step shorter: its four products take 280 clocks at any width up to 128 columns
// (measured; 537 at 256), 16 KB of weights in 0.15 us, twice what an SM's share
// of the memory brings in that time. Few units are split over K instead.
//
// Prompts (tiles of 256 tokens): a pair of CTAs makes one product of 256 rows,
// each holding 128 rows of the weights and half of the tokens (cta_group::2). A
// k-step then brings an SM 32 KB instead of 48 and the ring holds 6 steps instead
// of 4 (T=8192 E=8 k=2 H=I=2048: `down` 114 -> 100 us, `up` 178 -> 176).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace mr {

constexpr int kGemmThreads = 256;   // warp 0 weights, 1 products, 2 tokens, 3 spare, 4-7 epilogue
constexpr int kEpilogueThreads = 128;
constexpr int kMaxStages = 16;
constexpr int kRows = 128;          // weight rows of a CTA's unit
constexpr int kPairColumns = 256;   // tiles of this many tokens are taken by pairs of CTAs
constexpr int kStepBytes = 128;     // one row of a k-step
constexpr int kStepK = 64;

// ---- barriers --------------------------------------------------------------------------------------------------

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// One lane of a converged warp. Instructions of the tensor path take their
// operands from uniform registers; under this predicate the compiler knows that
// a single thread runs them, while `lane == 0` makes it loop over the lanes for
// each (T=1 E=256 k=8, with time stamps: 350 ns a k-step of four products, 256
// under the predicate).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// One attempt without a suspend-time hint: 15 clocks on a complete phase, where
// mbar_try_wait takes 50 and holds up the copies or products issued after it
// (measured: 267 clocks a k-step of four products with it, 156 without).
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait of one role: false, with the CTA's `gone` word raised, if it
// gave up or another role did. Every role leaves its loops then.
struct Waits {
    volatile int* gone;
    uint32_t tries;

    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const
    {
        for (int i = 0; i < 64; ++i)  // the usual case: complete, or about to be
            if (mbar_poll(bar, parity)) return true;
        for (uint32_t i = 0; i < tries; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*gone) return false;
        }
        *gone = 1;
        return false;
    }
};

// The epilogue's wait: one thread polls and all 128 learn its answer at a
// barrier (so none leaves alone). All polling, four warps slow the waits of the
// roles that feed the products (the same barrier unit): 190 ns a k-step.
__device__ __forceinline__ bool epilogue_wait(const Waits& wait, uint64_t* bar, uint32_t parity)
{
    uint32_t mine = 1;
    if (threadIdx.x == kGemmThreads - kEpilogueThreads) {
        mine = wait(bar, parity) ? 1 : 0;
        asm volatile("tcgen05.fence::after_thread_sync;\n\ttcgen05.fence::before_thread_sync;" ::: "memory");
    }
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(mine)
        : "memory");
    return all != 0;
}

// Position in the ring of stages: the stage and how often the ring wrapped.
struct RingPos {
    int s = 0;
    uint32_t wraps = 0;

    __device__ __forceinline__ void next(int stages)
    {
        if (++s == stages) {
            s = 0;
            ++wraps;
        }
    }
};

// The cluster address of this variable in CTA `rank`, and an arrival at a barrier there.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A named barrier of the epilogue warps.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// ---- tensor copies -----------------------------------------------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

__device__ __forceinline__ void load_box3(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void load_box2(uint32_t dst, const CUtensorMap* m, int x, int y, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// The same for a pair of CTAs: into this CTA's memory, counted by a barrier of
// either one (a cluster address).
__device__ __forceinline__ void load_box3_pair(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void load_box2_pair(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Four rows of a matrix, one after the other in shared memory (the map's box is one row).
__device__ __forceinline__ void load_rows4(uint32_t dst, const CUtensorMap* m, int x, int4 r, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(m), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_addr(bar))
        : "memory");
}

// ---- tensor memory and products ----------------------------------------------------------------------------------

// All lanes of one warp (PAIR: of one warp in each CTA); `slot` (shared) receives the address.
template <bool PAIR = false>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t columns)
{
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        return;
    }
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

template <bool PAIR = false>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    if (PAIR) {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
        return;
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand of 128-byte swizzled rows, K contiguous: 8 rows of 128
// bytes make an atom, atoms follow one another every 1024 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// bf16 x bf16 -> fp32, 128 rows (a pair's: 256), n columns (a multiple of 16; a
// pair's: of 32), both operands K-major.
__device__ __forceinline__ uint32_t product_desc(int n, bool pair = false)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((pair ? 16u : 8u) << 24);
}

// D (+)= A B^T over 16 of K. PAIR: issued by the pair's first CTA for both; each
// has its rows of A, its half of B's rows and its rows of D at these addresses.
template <bool PAIR = false>
__device__ __forceinline__ void mma16(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add)
{
    if (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u)
            : "memory");
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(add ? 1u : 0u)
        : "memory");
}

// `bar` is arrived at when all products issued so far by this thread are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// The same for a pair's products, at this barrier of the CTAs in `mask`.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar, uint16_t mask)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(mask)
        : "memory");
}

// 16 consecutive columns of this warp's 32 rows: the lane's row.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// ---- shared memory of a CTA ----------------------------------------------------------------------------------------

struct GemmBars {
    uint64_t full[kMaxStages];   // a stage's weights and tokens are there (one arrival each, and their bytes)
    uint64_t empty[kMaxStages];  // the products have read it
    uint64_t acc_full[2];        // an accumulator is complete
    uint64_t acc_empty[2];       // the epilogue has read it
    uint64_t drained;            // every product issued is done
    int cols[kMaxStages];        // columns of the unit that starts in this stage
    uint32_t tmem;
    int gone;
};

// The products' wait for stages, asked one stage ahead: the answer comes while
// the products of the stage before are issued (56 clocks a step less).
struct StagePoll {
    bool there = false;

    // Waits for the stage at `pos` and asks for the one after it.
    __device__ __forceinline__ bool take(const Waits& wait, GemmBars& bars, RingPos pos, int stages)
    {
        if (!there && !wait(&bars.full[pos.s], pos.wraps & 1)) return false;
        pos.next(stages);
        there = mbar_poll(&bars.full[pos.s], pos.wraps & 1);
        return true;
    }
};

}  // namespace mr
