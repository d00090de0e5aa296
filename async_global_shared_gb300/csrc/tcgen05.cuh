// The fifth-generation tensor core's instructions (tcgen05) as the 8-bit
// matrix product uses them: tensor memory, one-thread matrix instructions on
// shared-memory operands, and accumulator loads.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace ap {
namespace ptx {

// CG is the instructions' CTA group: 1, or 2 for a pair of CTAs (cluster ranks
// 2i and 2i + 1) that share one matrix instruction. A kernel uses one of them
// throughout.

// Allocate `cols` columns of tensor memory (a power of two, 32..512); the
// address goes to shared memory at dst. Executed by one whole warp (of each
// CTA of a pair).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Descriptor of a K-major operand in shared memory: rows of 128 bytes in the
// 128-byte swizzle, eight rows (1024 bytes) a swizzle atom, atoms one after
// another; addr 1024-byte aligned (plus 32 bytes for each k step inside the
// atom). Bits 0-13 address / 16, 16-29 leading offset / 16 (not used by a
// swizzled K-major operand), 32-45 stride between atoms / 16, 46-48 version 1,
// 61-63 swizzle mode 2 (128 bytes).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: e4m3 x e4m3 into 32-bit floats, both operands
// K-major, an M x N tile. Bits 4-5 accumulator type 1 (float), 7-9 and 10-12
// operand types 0 (e4m3), 17-22 N / 8, 24-28 M / 16.
__host__ __device__ constexpr uint32_t e4m3_instr_desc(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n / 8) << 17) | (static_cast<uint32_t>(m / 16) << 24);
}

// d (tensor memory) = a * b^T, or += where accumulate: one k step of 32
// values. Issued by one thread (of a pair's even CTA); completes
// asynchronously. In a pair each CTA holds half of a's rows, half of b's rows
// and, in its own tensor memory, the results of its half of a's rows.
template <int CG>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
            : "memory");
}

// Arrive on bar (of both CTAs of a pair) once every matrix instruction this
// thread issued so far has completed (its operands read, its results in tensor
// memory).
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}

// As tensor_g2s_2d; in a pair `bar` may be the other CTA's (a cluster address).
template <int CG>
__device__ __forceinline__ void operand_g2s(uint32_t dst, const void* tmap, int32_t c0, int32_t c1, uint32_t bar) {
    if constexpr (CG == 1)
        tensor_g2s_2d(dst, tmap, c0, c1, bar);
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%2, %3}], [%4];" ::"r"(dst),
            "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}

// Values in the shared memory of a CTA of the cluster (address from mapa).
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Consecutive columns of the calling warp's 32 lanes: lane l, column i goes to
// v[i] of thread l. The values are there after tmem_wait_ld. Naming their
// registers there would keep their uses behind it, but costs a move a value
// (as many instructions as the sums); their uses are fma_ordered instead, which
// as volatile as the wait stay behind it. (Loads from memory may cross it.)
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;"); }
__device__ __forceinline__ float fma_ordered(float a, float b, float c) {
    float r;
    asm volatile("fma.rn.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr));
}

// One thread of the warp, the same one every time; the compiler knows that
// what it guards runs once for the warp, which makes issuing matrix
// instructions and copies several times cheaper than under "lane == 0".
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Whether a barrier's phase has completed, without the suspension of
// mbar_try_wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Arrive where `yes`, without a branch. REMOTE: on another CTA's barrier (an
// address from mapa), relaxed: what it signals, reads of tensor memory, has
// completed by tmem_wait_ld and is ordered by tcgen05_fence_before.
template <bool REMOTE>
__device__ __forceinline__ void mbar_arrive_if(bool yes, uint32_t bar) {
    if constexpr (REMOTE)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
            "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
            "r"(static_cast<uint32_t>(yes))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
            "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
            "r"(static_cast<uint32_t>(yes))
            : "memory");
}

// Registers of this warpgroup's threads, out of what the CTA was launched with.
template <int N>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Shared -> global store of one 2-D box into a tensor map's matrix; what lies
// outside the matrix is not written. Tracked by bulk groups.
__device__ __forceinline__ void tensor_s2g_2d(const void* tmap, int32_t c0, int32_t c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap), "r"(c0),
                 "r"(c1), "r"(src)
                 : "memory");
}

}  // namespace ptx
}  // namespace ap
