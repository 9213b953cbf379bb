// Product in 8-bit integers for up to four token rows of a group: every weight byte goes from memory into a register once and
// meets all tokens there (four products an instruction).  Nothing but the launch stands before the weights' loads: no tensor
// memory, no conversion, and of one token's plain product no second kernel for its rounding.
//
// A warp has R weight rows at a time, a lane 16 bytes of every 512, U of those steps on their way while the U before them
// are multiplied.  The tokens lie in shared memory as 8-bit integers; R rows share what a lane reads of them.
//
// Bound by memory where the weights are large (8 sorted rows of 8 experts of 4096 x 7168 38.5 us, 6.1 TB/s; 1 x 12288 x 7168 18 with its
// rounding), by the launch and two trips to memory where they are small (1 x 2112 x 7168 6.3 us, 5.1 without rounding).
#include <atomic>

#include "device.h"
#include "int8.cuh"
#include "launch.h"
#include "sorted.h"

namespace mse {
namespace sorted {
namespace {

constexpr int kFewThreads = 256, kWarps = kFewThreads / 32;
constexpr int kStep = 512;   // bytes of a row that a warp reads at once

// 16 bytes of weights, the ones behind K 0
__device__ __forceinline__ uint4 load16(const int8_t *row, int64_t k, int64_t K) {
    if (k + 16 <= K) return __ldcs(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K) w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (i % 4 * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sums of v[0 .. M) over the warp, M a power of two: lane l has that of v[l >> (5 - log2 M)].
template <int M>
__device__ __forceinline__ int warp_sums(int (&v)[M], int lane) {
    int d = 16;
#pragma unroll
    for (int m = M; m > 1; m /= 2, d /= 2) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < m / 2; ++i) {
            const int mine = up ? v[i + m / 2] : v[i], other = up ? v[i] : v[i + m / 2];
            v[i] = mine + __shfl_xor_sync(~0u, other, d);
        }
    }
    for (; d > 0; d /= 2) v[0] += __shfl_xor_sync(~0u, v[0], d);
    return v[0];
}

struct FewParams {
    Int8Gemm g;
    const void *x; int64_t ldx;      // ROUND: tokens in bf16 or fp32
    int f32, x_wide;                 // x_wide: token rows (of either kind) begin at multiples of 16 bytes
    int weights_early;               // a kernel of the same call came before: weights and offsets are complete
};

// TM: token rows of a tile
template <int TM, int R, int U, bool ROUND>
__global__ void __launch_bounds__(kFewThreads, 2) int8_few_kernel(const FewParams p) {
    extern __shared__ __align__(16) uint8_t few_smem[];   // [TM][pitch] tokens
    __shared__ uint32_t tops[TM][kWarps];
    __shared__ float scale_s[TM];
    const Int8Gemm &g = p.g;
    const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(~0u, tid / 32, 0);
    const int64_t pitch = (g.K + kStep - 1) / kStep * kStep;
    if (!p.weights_early) pdl_wait();
    RowTile t;
    if (!row_tile(g.offsets, g.groups, g.T, TM, blockIdx.y, t)) {
        if (p.weights_early) pdl_wait();
        return;
    }
    const int8_t *weights = g.wq + (int64_t)t.group * g.N * g.ldw;
    const int64_t row_groups = (g.N + R - 1) / R, stride = (int64_t)gridDim.x * kWarps;
    const int steps = (int)((pitch / kStep + U - 1) / U);
    auto load = [&](int64_t group, int step, uint4 (&w)[R][U]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = group * R + r;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t k = ((int64_t)step * U + u) * kStep + lane * 16;
                w[r][u] = n < g.N && k < g.K ? load16(weights + n * g.ldw, k, g.K) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    int64_t group = (int64_t)blockIdx.x * kWarps + warp;
    uint4 now[R][U];
    if (group < row_groups) load(group, 0, now);

    // ---- the tokens, while the first weights are on their way
    if (p.weights_early) pdl_wait();
    if constexpr (ROUND) {
        auto value8 = [&](int row, int64_t k, float (&v)[8]) {
            const int64_t at = (t.row0 + row) * p.ldx + k;
            if (p.f32) {
                const float *x = static_cast<const float *>(p.x) + at;
                if (p.x_wide && k + 8 <= g.K) {
                    const float4 a = reinterpret_cast<const float4 *>(x)[0], b = reinterpret_cast<const float4 *>(x)[1];
                    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = k + i < g.K ? x[i] : 0.f;
                }
            } else {
                const uint16_t *x = static_cast<const uint16_t *>(p.x) + at;
                if (p.x_wide && k + 8 <= g.K) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(x);
                    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] = __uint_as_float(u[i] << 16);
                        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = k + i < g.K ? bf16_bits_to_f32(x[i]) : 0.f;
                }
            }
        };
#pragma unroll
        for (int r = 0; r < TM; ++r) {
            uint32_t top = 0;
            if (r < t.rows)
                for (int64_t k = (int64_t)tid * 8; k < g.K; k += kFewThreads * 8) {
                    float v[8];
                    value8(r, k, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
                }
            top = __reduce_max_sync(~0u, top);
            if (lane == 0) tops[r][warp] = top;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < TM; ++r) {
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = max(top, tops[r][w]);
            const RowScale s = row_scale(top);
            if (tid == 0) scale_s[r] = s.scale;
            for (int64_t k = (int64_t)tid * 8; k < pitch; k += kFewThreads * 8) {
                uint32_t b[4] = {0, 0, 0, 0};
                if (r < t.rows && k < g.K && !s.nan) {
                    float v[8];
                    value8(r, k, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t m = int8x2_of(v[2 * i], v[2 * i + 1], s);
                        b[i] = __byte_perm((uint32_t)m, (uint32_t)(m >> 32), 0x0040);
                    }
                }
                *reinterpret_cast<uint2 *>(few_smem + r * pitch + k) =
                    make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < TM; ++r) {
            const int8_t *x = g.xq + (int64_t)(t.row0 + r) * g.ldx;
            for (int64_t k = (int64_t)tid * 16; k < pitch; k += kFewThreads * 16) {
                uint32_t b[4] = {0, 0, 0, 0};
                if (r < t.rows && p.x_wide && k + 16 <= g.K) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(x + k);
                    b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
                } else if (r < t.rows) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (k + i < g.K) b[i / 4] |= (uint32_t)(uint8_t)x[k + i] << (i % 4 * 8);
                }
                *reinterpret_cast<uint4 *>(few_smem + r * pitch + k) = make_uint4(b[0], b[1], b[2], b[3]);
            }
            if (tid == 0) scale_s[r] = r < t.rows ? g.xs[t.row0 + r] : 0.f;
        }
    }
    __syncthreads();

    int acc[R * TM];
#pragma unroll
    for (int i = 0; i < R * TM; ++i) acc[i] = 0;
    for (int step = 0; group < row_groups;) {
        const bool last = step + 1 == steps;
        const int64_t then = last ? group + stride : group;
        uint4 next[R][U];
        if (then < row_groups) load(then, last ? 0 : step + 1, next);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = ((int64_t)step * U + u) * kStep + lane * 16;
            if (k < pitch) {   // the same for the warp
#pragma unroll
                for (int c = 0; c < TM; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(few_smem + c * pitch + k);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        int &a = acc[r * TM + c];
                        a = __dp4a((int)now[r][u].x, (int)x.x, a);
                        a = __dp4a((int)now[r][u].y, (int)x.y, a);
                        a = __dp4a((int)now[r][u].z, (int)x.z, a);
                        a = __dp4a((int)now[r][u].w, (int)x.w, a);
                    }
                }
            }
        }
        if (last) {
            constexpr int M = R * TM, kShift = M == 1 ? 5 : M == 2 ? 4 : M == 4 ? 3 : M == 8 ? 2 : M == 16 ? 1 : 0;
            const int sum = warp_sums<M>(acc, lane), i = lane >> kShift, c = i % TM;
            const int64_t n = group * R + i / TM;
            if ((lane & ((1 << kShift) - 1)) == 0 && n < g.N && c < t.rows) {
                const float y = (float)sum * scale_s[c] * g.ws[(int64_t)t.group * g.N + n];
                const int64_t at = (int64_t)(t.row0 + c) * g.N + n;
                if (g.out_f32)
                    static_cast<float *>(g.out)[at] = y;
                else
                    static_cast<uint16_t *>(g.out)[at] = f32_to_bf16_bits(y);
            }
#pragma unroll
            for (int j = 0; j < M; ++j) acc[j] = 0;
            step = 0;
        } else {
            ++step;
        }
        group = then;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) now[r][u] = next[r][u];
    }
}

template <int TM, int R, int U, bool ROUND>
cudaError_t run(const FewParams &p, int slots, int sm_count, bool pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done;   // bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(done.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(int8_few_kernel<TM, R, U, ROUND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kInt8FewBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(1ull << (dev & 63), std::memory_order_acq_rel);
    }
    const int64_t warps = (p.g.N + R - 1) / R, ctas = (warps + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)std::min<int64_t>(ctas, std::max<int64_t>(1, (2 * sm_count + slots - 1) / slots)), (unsigned)slots);
    const size_t smem = (size_t)TM * (size_t)((p.g.K + kStep - 1) / kStep * kStep);
    return launch_kernel(int8_few_kernel<TM, R, U, ROUND>, grid, kFewThreads, smem, pdl, 1, s, p);
}

// One weight row at a time while the rows last for every warp of the grid once, two, which share what is read of the tokens, from
// twice as many on.  (us with one and two: 4 x 2112 x 7168 7.4, 7.7; 4 x 12288 x 7168 23.3, 20.2; 2 x 7168 x 6144 10.9, 11.0.)
cudaError_t run_rows(const FewParams &p, int tile_rows, int slots, int sm_count, bool pdl, cudaStream_t s) {
    const bool two = p.g.N * slots >= 4 * (int64_t)sm_count * kWarps;
    switch (tile_rows) {
        case 1: return p.x ? run<1, 1, 8, true>(p, slots, sm_count, pdl, s) : run<1, 1, 8, false>(p, slots, sm_count, pdl, s);
        case 2: return two ? run<2, 2, 4, false>(p, slots, sm_count, pdl, s) : run<2, 1, 8, false>(p, slots, sm_count, pdl, s);
        default: return two ? run<4, 2, 4, false>(p, slots, sm_count, pdl, s) : run<4, 1, 8, false>(p, slots, sm_count, pdl, s);
    }
}

}  // namespace

bool int8_few_serves(int tile_rows, int64_t K) { return tile_rows <= 4 && tile_rows * ((K + kStep - 1) / kStep * kStep) <= kInt8FewBytes; }

cudaError_t launch_int8_few(const Int8Gemm &g, int tile_rows, const void *x, int f32, int64_t ldx, bool weights_early, int sm_count,
                            bool pdl, cudaStream_t s) {
    FewParams p;
    p.g = g;
    p.x = x; p.ldx = ldx; p.f32 = f32;
    const uintptr_t bits = x ? reinterpret_cast<uintptr_t>(x) | (uintptr_t)ldx * (f32 ? 4 : 2)
                             : reinterpret_cast<uintptr_t>(g.xq) | (uintptr_t)g.ldx;
    p.x_wide = bits % 16 == 0;
    p.weights_early = weights_early;
    const int64_t per = (g.T + tile_rows - 1) / tile_rows;
    const int slots = (int)(g.offsets ? std::min<int64_t>(g.T, g.T / tile_rows + std::min<int64_t>(g.groups, g.T)) : per);
    return run_rows(p, tile_rows, slots, sm_count, pdl, s);
}

}  // namespace sorted
}  // namespace mse
