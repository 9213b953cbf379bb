// Pieces shared by the tensor-core kernels of the products in 8-bit integers.
//
// sm_103a's tensor cores have no 8-bit integer kind.  Every 8-bit integer is a value of fp16, a product of two is below 2^14 + 1
// and a sum of 1024 of them at most 2^24, so that kind::f16 sums kChunkBlocks k-blocks exactly in its fp32 accumulator; the chunks
// are then added as 32-bit integers.  The weights' bytes become fp16 on their way from shared memory to tensor memory, where
// the MMA takes them as its A operand: memory and L2 move one byte a weight, and shared memory is read once by the conversion
// and not by the MMA.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "int8.cuh"
#include "sorted.h"

namespace mse {
namespace sorted {

constexpr int kInner = 128;                          // k of a block
constexpr int kChunkBlocks = 8;                      // k-blocks to an exact sum
constexpr uint32_t kWeightTile = 128 * kInner;       // bytes: 128 rows
constexpr uint32_t kATmem = kInner / 2;              // TMEM columns of a k-block of weights in fp16

// Instruction descriptor, kind::f16: D fp32 ([4,6) = 1), A and B fp16 ([7,10) = [10,13) = 0), both K-major, N >> 3 at [17,23),
// M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] B[smem]^T over 16 values of k
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 16 columns from registers to tensor memory
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 8 columns from tensor memory
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four 8-bit integers to four fp16: 0x64 over the byte v + 128 is 1152 + v, whose difference to 1152 is exact.
__device__ __forceinline__ void half_of_bytes(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off), y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// One warp's 32 weight rows of a k-block (128 bytes each, 128-byte swizzle) from shared to tensor memory as fp16.  (All of a
// row's bytes first, and the next k-block's while these go to tensor memory, makes the products 5 to 15% slower.)
__device__ __forceinline__ void convert_rows(const uint8_t *tile, int row, uint32_t taddr) {
    const uint8_t *mine = tile + row * kInner;
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 w = *reinterpret_cast<const uint4 *>(mine + (((c + i) ^ (row & 7)) * 16));
            half_of_bytes(w.x, h[8 * i], h[8 * i + 1]);
            half_of_bytes(w.y, h[8 * i + 2], h[8 * i + 3]);
            half_of_bytes(w.z, h[8 * i + 4], h[8 * i + 5]);
            half_of_bytes(w.w, h[8 * i + 6], h[8 * i + 7]);
        }
        tmem_st16(taddr + c * 8, h);
    }
}

// The one lane of a converged warp that issues tensor-core and TMA instructions (see fp8_tc.cuh on why the warp runs the loop
// around them together).
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Bounded wait by a whole warp: true when every lane saw the phase complete.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag, const Int8Gemm &g) {
    return __all_sync(~0u, mbar_wait_bounded(bar, parity, abort_flag, g.wait_limit_ns, g.err));
}
__device__ __forceinline__ uint64_t drain_limit_of(uint64_t wait_limit_ns) {
    return wait_limit_ns > 100000000ull ? wait_limit_ns : 100000000ull;
}

// Arrive on an mbarrier of a CTA of the cluster without ordering memory: it announces that TMEM was read (tcgen05.wait::ld and a
// tcgen05 fence order that).  A release at cluster scope would wait for the thread's stores of the tile before.
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The same with the release that an arrival has by default, of the CTA's scope: for what went to TMEM (tcgen05.wait::st and a
// tcgen05 fence order it; a release at cluster scope takes several hundred cycles for every k-block).
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 16 bytes to shared memory of a CTA of the cluster
__device__ __forceinline__ void st_cluster_s32x4(uint32_t addr, int4 v) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

}  // namespace sorted
}  // namespace mse
