// w4a4_pair.cuh -- what the 4-bit products on CTA pairs share (gemm_w4a4_tile.cu,
// gemm_moe.cu): shared memory and TMEM of a tile; and for all products on pairs
// the wrappers of the instructions that work on both CTAs.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace nvfp4 {

using namespace sm100;

constexpr int kTlEpiWarps = 8;
constexpr int kTlThreads = 32 * (kTlEpiWarps + 2);  // + copies, MMA
constexpr int kTlStoreBytes = 2048;                  // a warp's staging for TMA stores: 32 rows of 64 bytes

template <bool kNv, int BN>
struct TlShape {
    static constexpr int kTiles = kNv ? 4 : 2;                 // scale tiles per stage and 128 rows
    static constexpr int kBRowTiles = (BN + 127) / 128;         // scale tiles over B's rows
    static constexpr int kABytes = 128 * 128, kBBytes = BN / 2 * 128;
    static constexpr int kSaBytes = kTiles * 512, kSbBytes = kBRowTiles * kTiles * 512;
    static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
    static constexpr int kFixed = kTlEpiWarps * kTlStoreBytes + 512;
    static constexpr int kFit = (232448 - kFixed) / kStageBytes;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr size_t kSmem = kFixed + (size_t)kStages * kStageBytes;
    static constexpr int kSfA = kTiles * 4, kSfB = kTiles * kBRowTiles * 4, kSf = kSfA + kSfB;
    static constexpr int kTmemCols = 512;
    // columns: accumulator 0 at 0, accumulator 1 at BN - kShared, then two stages' scales (more would take
    // columns from the accumulators: 343 us instead of 334 at 16384 x 18944 x 3584)
    static constexpr int kSfBufs = 2;
    static constexpr int kOver = 2 * BN + kSfBufs * kSf - kTmemCols;
    static constexpr int kShared = kOver > 64 ? (kOver + 31) / 32 * 32 : kOver > 0 ? 64 : 0;
    static constexpr int kAcc1 = BN - kShared, kSfCol = 2 * BN - kShared;
    static_assert(kSfCol + kSfBufs * kSf <= kTmemCols && kSfBufs < kStages && (kShared == 0 || kShared >= 64),
                  "TMEM; each half of the epilogue has a shared chunk");
};

__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

// Loads whose bytes are counted on the pair leader's barrier.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(smem_addr(dst)),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"((uint64_t)map),
                 "r"(smem_addr(src)), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Arrival on a barrier of the pair.  What it hands over is TMEM that has been
// read (tcgen05.wait::ld), so a release of this thread's memory operations at
// cluster scope is not needed; it would wait for the stores in flight (1500
// cycles between two tiles).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool kBlock16>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    if (kBlock16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
            : "memory");
}

// D[tmem] (+)= A[smem] B[smem]^T over 16 elements of K, f16 or bf16 operands.
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One arrival on the barrier at bar's offset in both CTAs when the MMAs (and
// scale copies) issued so far have completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace nvfp4
