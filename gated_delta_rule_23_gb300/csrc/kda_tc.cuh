// What the kernels on the 5th-generation tensor cores share: bf16 products, swizzled descriptors, reads and writes of tensor memory,
// tensor-map copies, and blocks taken over from the grid.
#pragma once

#include <cuda.h>

#include "kda_device.cuh"

namespace kda {

// ---------------------------------------------------------------- tensor cores and copies
// 128-byte swizzled shared-memory matrix descriptors, as their two words.  K-major: groups of 8 rows 1024 bytes apart;
// MN-major: groups of 8 along K 1024 bytes apart, blocks of 64 along MN `lbo` apart.  The high word is the same for all;
// in the low one a step along the operand is an addition, so that the issuing thread spends an instruction or two a
// product (building whole descriptors there cost as much as the products themselves).
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
// (In a cluster a shared-memory address has the CTA's rank above its 18 bits.)
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr & 0x3ffff) >> 4) | ((lbo >> 4) << 16); }
// fp32 accumulator, bf16 A and B, A K-major, B K-major or (mn) MN-major
__device__ __forceinline__ constexpr uint32_t idesc_bf16(int M, int N, bool mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t A_MN = 1u << 15;   // with it A is MN-major too
// D[tmem] (+)= A B^T, A in shared or tensor memory, B in shared memory; ACC: added to D, else as `acc` says
template <bool ACC> __device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, int acc)
{
    if (ACC)
        asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.eq.u32 p, 0, 0;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}"
                     ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(DESC_HI) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}"
                     ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(DESC_HI), "r"(acc) : "memory");
}
template <bool ACC> __device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, int acc)
{
    if (ACC)
        asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.eq.u32 p, 0, 0;\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}"
                     ::"r"(d), "r"(a_tmem), "r"(b), "r"(idesc), "r"(DESC_HI) : "memory");
    else
        asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %4};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}"
                     ::"r"(d), "r"(a_tmem), "r"(b), "r"(idesc), "r"(DESC_HI), "r"(acc) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar) : "memory");
}

// 32 or 64 columns of the warp's 32 lanes, one row a thread: the load and the wait for it, as one statement so that no register
// is moved or spilled in between.
#define REGS8(k, a, i) k(a[i]), k(a[i + 1]), k(a[i + 2]), k(a[i + 3]), k(a[i + 4]), k(a[i + 5]), k(a[i + 6]), k(a[i + 7])
__device__ __forceinline__ void tmem_read32(uint32_t addr, float (&s)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;"
                 : REGS8("=&f", s, 0), REGS8("=&f", s, 8), REGS8("=&f", s, 16), REGS8("=&f", s, 24)
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_read64(uint32_t addr, float (&s)[2][32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
                 " tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
                 "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n tcgen05.wait::ld.sync.aligned;"
                 : REGS8("=&f", s[0], 0), REGS8("=&f", s[0], 8), REGS8("=&f", s[0], 16), REGS8("=&f", s[0], 24),
                   REGS8("=&f", s[1], 0), REGS8("=&f", s[1], 8), REGS8("=&f", s[1], 16), REGS8("=&f", s[1], 24)
                 : "r"(addr), "r"(addr + 32) : "memory");
}
#undef REGS8
// tcgen05.st of 32 columns without the wait for its completion
__device__ __forceinline__ void tmem_put32(uint32_t addr, const uint32_t (&u)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(addr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
                   "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]),
                   "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]),
                   "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
                 : "memory");
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b)
{
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t x;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(x));
    return x;
}

// The next block of the grid that has not started, which then never will: asked for, its answer (16 bytes) goes to shared
// memory and completes on the barrier.  take_answer: the block's index, -1 when there was none.
__device__ __forceinline__ void ask_for_block(uint32_t answer, uint32_t mbar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(answer), "r"(mbar) : "memory");
}
__device__ __forceinline__ int take_answer(uint32_t answer)
{
    int x;
    asm volatile("{\n .reg .b128 a;\n .reg .pred p;\n .reg .b32 y, z, u;\n ld.shared.b128 a, [%1];\n mov.b32 %0, -1;\n"
                 " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n"
                 " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, u}, a;\n}"
                 : "=r"(x) : "r"(answer) : "memory");
    return x;
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps (looked up once).
cudaError_t encode_fn(EncodeTiled *fn);

}  // namespace kda
