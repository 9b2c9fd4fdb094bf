// tcgen05 primitives of the tile products in dcnv4_orthogonalize.cuh,
// dcnv4_predictor_backward.cuh and dcnv4_mx.cuh: shared-memory and instruction
// descriptors, tensor-memory allocation and reads, TMA tile copies. (The
// predictor's kernel keeps its own K-major subset in dcnv4_predictor.cuh.)
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "dcnv4_async.cuh"

namespace dcnv4 {
namespace tc {

// Shared-memory operand descriptors (version 1): start address, leading and
// stride byte offsets, layout code (0: no swizzle, 2: 128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc(unsigned saddr, unsigned lead, unsigned stride, unsigned layout) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(stride >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) |
           (static_cast<uint64_t>(layout) << 61);
}
// Rows of 128 bytes in 8-row atoms of 1024 bytes, 16-byte chunk j of row r at
// chunk j ^ (r mod 8) (the TMA's 128-byte swizzle). The same bytes serve as a
// K-major operand (a row holds 64 k of one M/N index; 16 k further: +32 bytes)
// and as an MN-major one (a row holds 64 M/N indexes of one k; 16 k further:
// two atoms, +2048 bytes). Such an operand is its descriptor's low word: start
// address and, in the upper half, the step to the next 64 M/N indexes of an
// MN-major operand (K-major: unused); `bytes` further on it is the word plus
// bytes / 16. The high word is the same for all of them.
__device__ __forceinline__ uint32_t sw128(unsigned saddr, unsigned lead = 16u) {
    return ((saddr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
}
constexpr uint32_t kSw128High = (1024u >> 4) | (1u << 14) | (2u << 29);

// Instruction descriptor of kind::f16, fp32 accumulators, M = 128.
constexpr uint32_t kFmtF16 = 0u, kFmtBf16 = 1u;
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t fmt, int n, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// A whole converged warp makes the call, with the same values in every lane
// (warp index, tensor-memory address and the like taken from uniform()); its
// one lane with `lead` set (lead_lane()) issues. What a product needs then
// stays in uniform registers: in a branch of one lane, whose values the
// compiler has to move there for every product, the issue of a 128 x 64 x 16
// product took 86 cycles, in this form 49 (what its operands' shared-memory
// reads take); a 128 x 128 x 16 one takes 65. a, b: operands as sw128() gives
// them.
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kSw128High), "r"(lead)
        : "memory");
}
// 1 in one lane of the (converged) warp, 0 in the others
__device__ __forceinline__ uint32_t lead_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// A bounded wait of a whole warp, with one answer. Where a warp's lanes go on to a vote, a __syncwarp or a
// barrier, a lane that gave up by itself would leave the others waiting there for it without a limit.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit_ns)) != 0;
}
// arrives on `bar` once every tcgen05 operation this thread issued so far has completed
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One whole warp allocates `cols` (a power of two, 32..512) columns.
__device__ __forceinline__ void alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// After a wait has given up, before the kernel leaves: what is still in flight is waited for, again with a limit,
// so that nothing lands in shared or tensor memory that is no longer this CTA's. The lane that loads: the last
// `depth` of `issued` steps, step k announced on full[k mod N]. The warp that issues products: all of them (the
// same lane is elected every time); `bar` is a barrier of one arrival for this alone.
template <int N>
__device__ __forceinline__ void drain_loads(uint64_t* full, long long issued, int depth) {
    for (long long k = issued > depth ? issued - depth : 0; k < issued; ++k)
        mbar_wait_bounded(&full[k % N], static_cast<unsigned>(k / N) & 1u, kCopyWaitLimitNs);
}
__device__ __forceinline__ void drain_products(uint64_t* bar) {
    if (lead_lane()) commit(bar);
    __syncwarp();
    warp_wait(bar, 0u, kCopyWaitLimitNs);
}

// 16 consecutive fp32 columns of this thread's lane; valid after wait_ld()
__device__ __forceinline__ void ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// TMA tile copies of a 3-D tensor map (no multicast); elements outside the
// tensor read as zeros and are not written.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int c0, int c1, int c2, const void* src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void bar_sync(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// barrier over `count` threads that also gives every one of them the AND of their `pred`s
__device__ __forceinline__ bool bar_and(int id, int count, bool pred) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %1, 0;\n\t"
        "bar.red.and.pred po, %2, %3, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(r)
        : "r"(pred ? 1u : 0u), "r"(id), "r"(count)
        : "memory");
    return r != 0;
}

}  // namespace tc
}  // namespace dcnv4
