// What the window attentions need of the tensor cores and the TMA besides
// tcgen05.cuh: matrix instructions issued by an elected lane of a whole warp,
// bf16 operands, TMEM loads in the layout of matrix fragments, 3-D boxes and
// boxes with an L2 policy.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "tcgen05.cuh"

namespace pa {

// 16 lanes x 32 columns in the layout of matrix fragments: of every 8 columns,
// r[4 i], r[4 i + 1] are columns 2 (lane % 4), + 1 of row lane / 4, r[4 i + 2],
// r[4 i + 3] the same of row lane / 4 + 8.
__device__ __forceinline__ void tmem_load_16x256b_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// idesc_f16_f32 for fp16 or bf16 operands (one type for both), A K-major.
__host__ __device__ constexpr uint32_t idesc_16_f32(int m, int n, bool b_mn_major, bool bf16)
{
    return idesc_f16_f32(m, n, b_mn_major) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10);
}

// umma_f16, umma_f16_ts and umma_commit for a whole warp that comes along
// together: only the lane whose `leader` is not 0 issues.  (The operands are
// then the same for the warp, which is what the instruction wants.)
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t leader;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(leader));
    return leader;
}

__device__ __forceinline__ void umma_f16_if(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(uint32_t(accumulate)), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void umma_f16_ts_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                               uint64_t b_desc, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(uint32_t(accumulate)), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void umma_commit_if(uint32_t leader, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

// Hint: fetch a tensor map that is a kernel parameter.
__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// tma_load_2d and tma_load_4d with an L2 eviction-priority policy.
__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d_hint(uint32_t dst, const CUtensorMap *map, int x0, int x1,
                                                 int x2, int x3, uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "l"(policy)
        : "memory");
}

// Box of a 3-D tensor map at (x0, x1, x2); x0 times the element size must be a
// multiple of 16 bytes.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x0, int x1, int x2,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x0), "r"(x1), "r"(x2)
        : "memory");
}

} // namespace pa
