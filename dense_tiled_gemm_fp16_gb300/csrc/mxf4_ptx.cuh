// Block-scaled MMA on MXFP4 operands: the tcgen05 forms the product and the
// mixture-of-experts kernels share.
#pragma once

#include <cstdint>

#include "mxf4_format.cuh"

namespace mxf4_dev {

// Limit of the waits that let work in flight end before a CTA gives up.
constexpr uint64_t kDrainNs = 1000000000ull;

// D[tmem] (+)= A * B with block scales; the two scales of each row's 64 values
// are the bytes 2 * half, 2 * half + 1 of the scale columns' words, `half` set
// in the instruction descriptor.
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// A 512-byte scale tile (32 rows of 16 bytes) to 4 tensor-memory columns, the
// same in each quarter of the lanes.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Unswizzled descriptor of a scale tile: 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(8) << 32) | (static_cast<uint64_t>(1) << 46);
}

// Instruction descriptor: e2m1 A and B (bits 7-9, 10-12), E8M0 scales (23),
// N / 8 (17-22), M / 128 (27-28), the scales' byte pair of B (4-5) and A (29-30).
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t m, uint32_t n, uint32_t half)
{
    return (1u << 7) | (1u << 10) | (1u << 23) | ((n >> 3) << 17) | ((m >> 7) << 27) | ((2 * half) << 4) |
           ((2 * half) << 29);
}

// Arrive on another CTA's barrier after tcgen05 loads that have completed, with
// tcgen05.fence::before_thread_sync between: nothing in memory is handed over, and
// a release would wait for the thread's own stores (1 000 to 1 800 cycles where a
// tile's last stores are in flight).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The forms of a CTA pair (one MMA over 256 rows, each CTA with its 128 rows of
// A, half the rows of B and the scales of its A rows and of all of B's).
__device__ __forceinline__ void umma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// (each CTA's tile, at the same offset in both, to its own tensor memory)
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 8 words of a lane to 8 columns of its tensor-memory lane.
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace mxf4_dev
