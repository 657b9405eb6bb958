// tcgen05 wrappers of the 8-bit integer path (kind::i8): int8 operands, int32
// accumulators.
#pragma once

#include "pair.cuh"

namespace patch {

// Instruction descriptor, kind::i8, both operands signed and K-major, D int32:
// D format bits 4-5 (2), A format 7-9 and B format 10-12 (1: signed), N>>3 at
// 17-22, M>>4 at 24-28, sparse flag bit 2.
__host__ __device__ constexpr uint32_t idesc_i8(int m, int n, bool sparse) {
    return (sparse ? (1u << 2) : 0u) | (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// The issuers run as whole warps in uniform control flow and let one elected lane
// issue (el: 1 on that lane). Inside a branch on the lane number, the same
// instructions cost one thread 360 to 400 cycles per 2:4 slab (metadata copy and two
// MMAs) instead of the 224 that the tensor pipe takes: their operands then have to be
// moved to uniform registers one by one.
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
#define PATCH_MMA_I8(NAME, GROUP)                                                                                     \
    __device__ __forceinline__ void NAME(uint32_t el, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, \
                                         uint32_t accumulate) {                                                        \
        asm volatile("{\n\t.reg .pred p, q;\n\t"                                                                      \
                     "setp.ne.b32 p, %4, 0;\n\t"                                                                      \
                     "setp.ne.b32 q, %5, 0;\n\t"                                                                      \
                     "@q tcgen05.mma." GROUP ".kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),                     \
                     "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(el)                                     \
                     : "memory");                                                                                      \
    }
#define PATCH_MMA_SP_I8(NAME, GROUP)                                                                                  \
    __device__ __forceinline__ void NAME(uint32_t el, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, \
                                         uint32_t e_tmem, uint32_t accumulate) {                                       \
        asm volatile("{\n\t.reg .pred p, q;\n\t"                                                                      \
                     "setp.ne.b32 p, %4, 0;\n\t"                                                                      \
                     "setp.ne.b32 q, %6, 0;\n\t"                                                                      \
                     "@q tcgen05.mma.sp." GROUP ".kind::i8 [%0], %1, %2, [%5], %3, p;\n\t}" ::"r"(d_tmem),            \
                     "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(e_tmem), "r"(el)                        \
                     : "memory");                                                                                      \
    }
PATCH_MMA_I8(mma_i8, "cta_group::1")
PATCH_MMA_I8(mma2_i8, "cta_group::2")
PATCH_MMA_SP_I8(mma_sp_i8, "cta_group::1")
PATCH_MMA_SP_I8(mma2_sp_i8, "cta_group::2")
#undef PATCH_MMA_I8
#undef PATCH_MMA_SP_I8
__device__ __forceinline__ void cp_el(uint32_t el, uint32_t taddr, uint64_t sdesc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::1.128x128b [%0], %1;\n\t}" ::"r"(taddr),
        "l"(sdesc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void cp2_el(uint32_t el, uint32_t taddr, uint64_t sdesc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::2.128x128b [%0], %1;\n\t}" ::"r"(taddr),
        "l"(sdesc), "r"(el)
        : "memory");
}
__device__ __forceinline__ void commit_el(uint32_t el, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(el)
        : "memory");
}
__device__ __forceinline__ void commit2_mask_el(uint32_t el, uint64_t* bar, uint16_t mask) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(mask), "r"(el)
        : "memory");
}

// 32 lanes x 8 columns of 32-bit.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr)
                 : "memory");
}

// One slab, on one CTA or (PAIR) on the CTA pair: 4 dense MMAs of K = 32, or 2
// sparse ones of K = 64, each with two of the four metadata columns at e_col, which
// are copied from behind the codes first. Operands advance by 32 bytes of A and 32
// (dense) or 64 (2:4) bytes of B per MMA.
template <bool PAIR>
__device__ __forceinline__ void issue_slab_i8(uint32_t el, bool sparse, bool first, uint32_t a_addr, uint32_t b_addr,
                                              uint32_t d_tmem, uint32_t e_col, uint32_t idesc_d, uint32_t idesc_s) {
    if (sparse) {
        const uint64_t ed = smem_desc(a_addr + kSparseValBytes, 16, 128, kLayoutNone);
        if (PAIR)
            cp2_el(el, e_col, ed);
        else
            cp_el(el, e_col, ed);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t ad = smem_desc(a_addr + i * 32, 16, 512, kLayoutSw64);
            const uint64_t bd = smem_desc(b_addr + i * 64, 16, 1024, kLayoutSw128);
            if (PAIR)
                mma2_sp_i8(el, d_tmem, ad, bd, idesc_s, e_col + 2 * i, !(first && i == 0));
            else
                mma_sp_i8(el, d_tmem, ad, bd, idesc_s, e_col + 2 * i, !(first && i == 0));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t ad = smem_desc(a_addr + i * 32, 16, 1024, kLayoutSw128);
            const uint64_t bd = smem_desc(b_addr + i * 32, 16, 1024, kLayoutSw128);
            if (PAIR)
                mma2_i8(el, d_tmem, ad, bd, idesc_d, !(first && i == 0));
            else
                mma_i8(el, d_tmem, ad, bd, idesc_d, !(first && i == 0));
        }
    }
}

}  // namespace patch
