// tc05.cuh -- fifth-generation tensor core (tcgen05) and TMEM helpers, sm_100 family.
//
// Conventions used by the tensor arm:
//  * One CTA, cta_group::1, M = 128 (the 128 weight rows of a tile) and
//    N = tokens of the tile.  A (the dequantised weights) lives in TMEM, B (the
//    activations) in shared memory, D (fp32) in TMEM.
//  * A TMEM address is (lane << 16) | column.  A warp may only touch the 32
//    lanes of its sub-partition (warp id % 4).
#pragma once

#include <cstdint>

namespace w4a16 {

// Instruction descriptor of tcgen05.mma .kind::f16: fp32 accumulate, bf16 A
// and B, both K-major, shape M x N.
__host__ __device__ constexpr uint32_t tc_idesc_bf16(int M, int N) {
    return (1u << 4)                       // D format: f32
           | (1u << 7)                     // A format: bf16
           | (1u << 10)                    // B format: bf16
           | (uint32_t(N >> 3) << 17)      // N / 8
           | (uint32_t(M >> 4) << 24);     // M / 16
}

// Shared-memory matrix descriptor for a K-major operand stored with the
// 128-byte swizzle: rows of 128 bytes, 8-row atoms of 1024 bytes (the layout a
// SWIZZLE_128B TMA load of a 64-element bf16 box writes).  The tile must start
// on a 1024-byte boundary; advancing K by 16 elements adds 32 bytes to the
// start address.
__device__ __forceinline__ uint64_t tc_sdesc_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFF);        // start address / 16
    d |= uint64_t(1) << 16;                          // leading byte offset (unused with swizzle)
    d |= uint64_t(1024 >> 4) << 32;                  // stride byte offset: 8 rows x 128 B
    d |= uint64_t(1) << 46;                          // descriptor version (sm_100)
    d |= uint64_t(2) << 61;                          // layout: 128-byte swizzle
    return d;
}

// Instruction descriptor bits: the operand lies along M (or N) instead of K.
constexpr uint32_t kTcAMajorM = 1u << 15;
constexpr uint32_t kTcBMajorN = 1u << 16;

// The same for rows of 64 bytes (32 elements of K) with the 64-byte swizzle:
// 8-row atoms of 512 bytes.
__device__ __forceinline__ uint64_t tc_sdesc_sw64(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFF);
    d |= uint64_t(1) << 16;
    d |= uint64_t(512 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(4) << 61;                          // layout: 64-byte swizzle
    return d;
}

// Shared-memory matrix descriptor for an operand that lies along M or N, with
// the 128-byte swizzle: each K index is a row of 128 bytes (64 elements of M or
// N), 8-row atoms of 1024 bytes.  `block_bytes`: from one block of 64 elements
// to the next.  Advancing K by 16 adds two atoms (2048 bytes) to the address.
__device__ __forceinline__ uint64_t tc_sdesc_sw128_mn(uint32_t smem_addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= uint64_t((smem_addr >> 4) & 0x3FFF);
    d |= uint64_t(block_bytes >> 4) << 16;           // leading byte offset: next 64 elements
    d |= uint64_t(1024 >> 4) << 32;                  // stride byte offset: next 8 of K
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

__device__ __forceinline__ void tc_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tc_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[tmem] . B[smem]^T ; accumulate when `acc` is nonzero.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}

// D[tmem] (+)= A[smem] . B[smem]^T ; accumulate when `acc` is nonzero.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrive once on an mbarrier when every tcgen05 operation this thread issued
// before has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// 16 lanes x 256 bits, 4 repetitions along columns: thread (g = lane/4,
// t = lane%4) supplies, for repetition r, {lane g: column 8r+2t, 8r+2t+1}
// and {lane g+8: column 8r+2t, 8r+2t+1} (the m16n8 accumulator pattern).
__device__ __forceinline__ void tc_st_16x256b_x4(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 bits, 32 repetitions: thread i gets columns c .. c+31 of lane i.
__device__ __forceinline__ void tc_ld_32x32b_x32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// 32 lanes x 32 bits, 8 repetitions: thread i gets columns c .. c+7 of lane i.
__device__ __forceinline__ void tc_ld_32x32b_x8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7])
        : "r"(taddr)
        : "memory");
}

}  // namespace w4a16
