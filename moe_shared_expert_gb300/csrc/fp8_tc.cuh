// Pieces shared by the tensor-core kernels of the block-scaled 8-bit products.
#pragma once
#include "common.cuh"
#include "fp8.cuh"
#include "routed.h"

namespace mse {
namespace routed {

constexpr uint32_t kOperandTile = 128 * 128;   // 128 rows x 128 bytes (one k-block), 128-byte swizzle

// Instruction descriptor, kind::f8f6f4: D fp32 [4,6) = 1, A and B e4m3 ([7,10) = [10,13) = 0), both
// K-major, N >> 3 at [17,23), M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem]^T over 32 e4m3 values of k
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on an mbarrier of a CTA of the cluster without ordering memory: what it announces is that
// TMEM was read (tcgen05.wait::ld and a tcgen05 fence order that).  A release at cluster scope here
// waits for the thread's outstanding global loads, once per k-block: 1.6 times the kernel's time.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 16 bytes to shared memory of a CTA of the cluster
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// The token tile of slot z: a dispatch's tile, or rows [z tile_rows, ..) of the one group.
__device__ __forceinline__ bool tile_of_slot(const BlockGemm &g, int z, Tile &t) {
    if (g.tiles) {
        if (z >= *g.n_tiles) return false;
        t = g.tiles[z];
    } else {
        t.row0 = z * g.tile_rows;
        t.rows = (int)min((int64_t)g.tile_rows, g.T - t.row0);
        t.expert = 0;
    }
    return true;
}

// The one lane of a converged warp that issues tensor-core and TMA instructions.  The warp runs the loop
// around them together, so that descriptors stay in uniform registers: issued from a region that one
// lane alone runs, each tcgen05.mma takes over 128 cycles to issue (670 instead of 512 cycles per k-block of 256 x 256).
__device__ __forceinline__ bool elect_lane() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Bounded wait by a whole warp: true when every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          const BlockGemm &g) {
    return __all_sync(~0u, mbar_wait_bounded(bar, parity, abort_flag, g.wait_limit_ns, g.err));
}

__device__ __forceinline__ uint64_t drain_limit(uint64_t wait_limit_ns) {
    return wait_limit_ns > 100000000ull ? wait_limit_ns : 100000000ull;
}

}  // namespace routed
}  // namespace mse
