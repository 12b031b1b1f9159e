// 5th-generation tensor core primitives (PTX tcgen05.*): tensor memory, the
// block-scaled FP4 matrix instruction, the 16-bit and FP8 ones for one CTA or a pair of
// CTAs, and their descriptors.
#pragma once

#include <cstdint>

#include "dh_common.cuh"

namespace dh {
namespace tc {

// Tensor memory: `cols` columns (a power of two, 32..512) of 128 lanes x 32 bits,
// allocated and freed by one whole warp; the address is written to *slot.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols));
}

// Order tcgen05 operations against thread synchronisation (mbarriers, barriers).
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive on an mbarrier once every tcgen05 operation that this thread issued is done.
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

// Shared-memory descriptor of an operand tile, K-major rows of 128 bytes with the
// 128-byte swizzle, 8-row groups 1,024 bytes apart: bits 0-13 address / 16, 16-29
// leading and 32-45 stride byte offset / 16, 46-48 version 1, 61-63 swizzle mode 2.
// A step along K inside the 128 bytes adds its bytes to the address.
__device__ __forceinline__ uint64_t desc_operand(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor of kind::mxf4nvf4, E2M1 operands (1 at bits 7 and 10),
// both K-major, UE4M3 scales (bit 23 = 0), N / 8 at bit 17, M / 16 at bit 24.
__host__ __device__ constexpr uint32_t idesc_nvf4(int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D (+)= sum over 4 blocks of 16 of scaleA scaleB A B, K = 64 per instruction. The
// scales are in tensor memory: row r's four (a 32-bit word) in lane r % 32 of
// column r / 32, the same in each group of 32 lanes.
__device__ __forceinline__ void mma_nvf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add ? 1u : 0u) : "memory");
}

// 8 columns of this warp's 32 lanes, as tmem_load16.
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}
// 16 columns of this warp's 32 lanes: thread l gets lane l's columns.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}
// 16 columns of this warp's 32 lanes, written from registers: lane l's columns from thread l.
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
                 :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                    "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------------
// One CTA (P = 1) or a pair (P = 2): in a pair, the CTAs of ranks 0 and 1 of a cluster
// share one output tile of 256 rows, 128 in each one's tensor memory; each holds its own
// 128 rows of A and half of the columns of B; rank 0 issues. A kernel uses one P throughout.
// ------------------------------------------------------------------------
template <int P>
__device__ __forceinline__ void tmem_alloc_of(uint32_t* slot, uint32_t cols) {
    if constexpr (P == 1) {
        tmem_alloc(slot, cols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int P>
__device__ __forceinline__ void tmem_free_of(uint32_t addr, uint32_t cols) {
    if constexpr (P == 1) tmem_free(addr, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols));
}

// Arrive on the barrier at this offset in every CTA of the tile once this thread's
// tcgen05 operations are done.
template <int P>
__device__ __forceinline__ void commit_all(uint64_t* bar) {
    if constexpr (P == 1) {
        commit(bar);
    } else {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
    }
}

// The same for this CTA's barrier alone.
template <int P>
__device__ __forceinline__ void commit_own(uint64_t* bar) {
    if constexpr (P == 1) commit(bar);
    else asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

// Operand whose rows run along M or N ("MN-major"): boxes of 128 bytes of M or N by
// `depth` rows of K, in the 128-byte swizzle; 8-row groups of K 1,024 bytes apart (the
// stride offset), boxes depth * 128 bytes (the leading offset). A step of s along K adds
// s * 128 bytes to the address.
__device__ __forceinline__ uint64_t desc_operand_mn(uint32_t addr, uint32_t depth) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(depth * 8) << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}

// Instruction descriptor of kind::f16 and kind::f8f6f4 with 32-bit accumulators (1 at bit
// 4): operand formats at bits 7 and 10 (f16 kind: 0 F16, 1 BF16; f8 kind: 0 E4M3), bits 15
// and 16 set for an MN-major A and B, N / 8 at bit 17, M / 16 at bit 24.
__host__ __device__ constexpr uint32_t idesc_f(int fmt, bool a_mn, bool b_mn, int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D (+)= A B over 32 bytes of K: 16 elements of 16 bits, 32 of 8.
template <int P, bool F8>
__device__ __forceinline__ void mma_f(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    const uint32_t on = add ? 1u : 0u;
    if constexpr (P == 1 && !F8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(on) : "memory");
    else if constexpr (P == 2 && !F8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(on) : "memory");
    else if constexpr (P == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(on) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(on) : "memory");
}

// 32 columns of this warp's 32 lanes (tmem_load_wait before the registers are read).
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

}  // namespace tc
}  // namespace dh
