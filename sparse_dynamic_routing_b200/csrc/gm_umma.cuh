// gm_umma.cuh - the sm_100a tensor-core, tensor-memory and tensor-copy primitives the dense
// refresh-edge and windowed-attention kernels use: tcgen05 MMA with its accumulator in tensor
// memory (TMEM), B in shared memory and A in either, TMEM allocation, loads and stores, and 3-d
// and 4-d tiled TMA copies. Inline PTX;
// the descriptor layouts follow the PTX ISA's tcgen05 "shared memory descriptor" and
// "instruction descriptor" tables (the bit positions are checked on the host against
// CUTLASS's definitions by tests/test_umma_desc.py).
#pragma once

#include <stdint.h>

namespace gm {
namespace umma {

// Instruction descriptor of tcgen05.mma kind::f16 with bf16 A and B, an fp32 accumulator,
// both operands K-major, dense, no negation: bits [4,6) D format (1 = f32), [7,10) A format
// (1 = bf16), [10,13) B format (1 = bf16), bits 15/16 A/B major (0 = K), [17,23) N / 8,
// [24,29) M / 16.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory matrix descriptor of a K-major operand in the 128-byte swizzle layout: rows of
// 128 bytes (64 bf16 along K), eight-row groups of 1024 bytes stacked along M/N, the group
// 1024-byte aligned. Fields: [0,14) start address / 16, [16,30) leading byte offset / 16
// (unused by swizzled K-major layouts; 1), [32,46) stride byte offset / 16 (1024 / 16 between
// eight-row groups), [46,48) version (1 on sm_100), [49,52) base offset (0: aligned groups),
// [61,64) layout (2 = 128-byte swizzle). A K step of 16 bf16 inside the 128-byte row advances
// the start address by 32 bytes.
__host__ __device__ constexpr uint64_t sdesc_sw128_kmajor(uint32_t smem_addr)
{
    return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The same descriptor with B held MN-major (bit 16): B's N runs along the contiguous dimension.
__host__ __device__ constexpr uint32_t idesc_bf16_f32_bmn(int M, int N) { return idesc_bf16_f32(M, N) | (1u << 16); }

#if defined(__CUDACC__)

// ---- MMA issue by a whole warp -----------------------------------------------------------------
//
// The functions below are executed by all lanes of a warp and act in the lane whose `lead` is not
// 0. Nothing branches on the lane, so operands that are the same in every lane stay in uniform
// registers, where the MMA instruction wants them: issued under `if (lane == 0)` each one first
// moves its descriptors there, 100 to 140 cycles per instruction instead of about 90, which a
// 128 x 128 x 16 product takes at the rate that cuBLAS reaches (64 at the nominal peak). Descriptors
// are given as their low word (sdesc_lo plus an offset in 16-byte units) and their high word, the
// same for every operand here.

__device__ __forceinline__ uint32_t elect_lead()
{
    uint32_t lead;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(lead));
    return lead;
}

// K-major operands: as sdesc_sw128_kmajor. MN-major ones: rows of 128 bytes hold 64 bf16 along M/N, one
// row per K index, eight-row groups of 1024 bytes stacked along K (the stride byte offset);
// block_bytes, the leading byte offset, leads from one 64-element block of M/N to the next. A K
// step of 16 advances the start address by 32 bytes K-major, by 2048 bytes MN-major.
constexpr uint32_t SDESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // as in sdesc_sw128_*
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t smem_addr, uint32_t block_bytes)
{
    return (smem_addr >> 4) | ((block_bytes >> 4) << 16);
}
constexpr uint32_t KMAJOR = 16;  // block_bytes of a K-major operand: the field reads 1

__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 da, db;\n mov.b64 da, {%2, %6};\n mov.b64 db, {%3, %6};\n"
        " setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %0, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%1], da, db, %4, p;\n}\n" ::"r"(lead),
        "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(SDESC_HI)
        : "memory");
}
// A in TMEM: lane = row of A, 32-bit column c = the bf16 pair (2c, 2c + 1) along K.
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 db;\n mov.b64 db, {%3, %6};\n"
        " setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %0, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], db, %4, p;\n}\n" ::"r"(lead),
        "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(SDESC_HI)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %0, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}\n" ::"r"(lead),
        "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         bool accumulate)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// Arrives (once) on the shared-memory barrier when every tcgen05 operation this thread issued
// before has completed.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

// A warpgroup's registers per thread, by all its warps; the others of the SM's share stay with the
// block, so all warpgroups together may take as many as the launch gave them.
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }

// Whole-warp TMEM allocation of `ncols` columns (a power of two >= 32); the base address is
// written to shared memory at `slot`.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(slot), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(base), "r"(ncols) : "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane (warp w of a warpgroup reads lanes
// 32 w .. 32 w + 31); completes at tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
        "[%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// The same for 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane written; completes at tmem_wait_st.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// The same for 16 columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// Waits for this thread's loads and makes the registers of one depend on it, so that nothing that
// uses them moves ahead of the wait while another load is already in flight.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }

// Tiled 3-d TMA load of one box into shared memory, completion counted on `bar`. The innermost
// coordinate x must be a multiple of 16 bytes' worth of elements.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Tiled 4-d TMA load of one box into shared memory, completion counted on `bar`; elements outside
// the tensor become zeros.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
// Tiled 4-d TMA store of one box from shared memory (elements outside the tensor are not
// written), its commit, and the wait until the committed stores have read their sources.
__device__ __forceinline__ void tma_store_4d(const void *tmap, uint32_t src, int x, int y, int z, int w)
{
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
// Makes this thread's shared-memory writes visible to the asynchronous proxy (TMA, tensor cores).
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

#endif  // __CUDACC__

}  // namespace umma
}  // namespace gm
