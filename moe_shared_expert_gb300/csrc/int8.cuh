// Rounding to 8-bit integers with one scale for each row, shared by the kernels that do it.
#pragma once
#include "common.cuh"

namespace mse {
namespace sorted {

constexpr float kInt8AmaxFloor = 7.888609052210118e-31f;   // 2^-100: scales stay normal numbers
constexpr float kLevels = 127.f;

// |v| as an integer that orders like the number, infinities and NaN above every finite value
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// A row's largest magnitude and what follows from it.
struct RowScale {
    float amax, inv, scale;   // inv = 127 / amax to within 2^-23
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    RowScale r;
    if (top >= 0x7F800000u) {   // infinity or NaN: the row stands for NaN
        r.amax = 1.f;
        r.inv = 0.f;
        r.scale = __uint_as_float(0x7FC00000u);
    } else {
        r.amax = fmaxf(__uint_as_float(top), kInt8AmaxFloor);
        r.inv = __fdiv_rn(kLevels, r.amax);
        r.scale = __fdiv_rn(r.amax, kLevels);
    }
    return r;
}

// rint(127 v / amax), ties to even, the quotient to nearest: 127 / 512 v first, so that nothing overflows; 512 is exact.
// The product with 127 / amax is within 2^-22 of the quotient's value, 2^-15 in all, so only near the middle of two integers does
// it take the division (every tie does; one value in a thousand of others).
__device__ __forceinline__ int int8_of(float v, const RowScale &r) {
    const float t = v * r.inv;
    const float n = rintf(t);
    if (fabsf(fabsf(t - n) - 0.5f) < 0.0009765625f && r.inv > 0.f)
        return (int)rintf(__fdiv_rn(v * (kLevels / 512.f), r.amax) * 512.f);
    return r.inv > 0.f ? (int)n : 0;
}

// silu(g) u
__device__ __forceinline__ float swiglu(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return g * r * u;
}

// The row tile of slot z: rows of one group.  Offsets are taken as they are in [0, T], so that no value of theirs leads out of
// the tensors.  Whole warps call it.
struct RowTile {
    int row0, rows, group;
};
__device__ __forceinline__ bool row_tile(const int32_t *offsets, int groups, int64_t T, int tile_rows, int64_t z, RowTile &t) {
    if (!offsets) {
        t.row0 = (int)(z * tile_rows);
        t.rows = (int)min((int64_t)tile_rows, T - z * tile_rows);
        t.group = 0;
        return t.rows > 0;
    }
    const int lane = threadIdx.x % 32;
    int64_t before = 0;   // tiles of the groups so far
    for (int g0 = 0; g0 < groups; g0 += 32) {
        const int g = g0 + lane;
        const int64_t a = g < groups ? min(max((int64_t)offsets[g], (int64_t)0), T) : 0;
        const int64_t b = g < groups ? min(max((int64_t)offsets[g + 1], (int64_t)0), T) : 0;
        const int64_t tiles = b > a ? (b - a + tile_rows - 1) / tile_rows : 0;
        int64_t upto = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += o;
        }
        const int64_t first = before + upto - tiles;
        const uint32_t owner = __ballot_sync(~0u, z >= first && z < first + tiles);
        if (owner) {
            const int from = __ffs(owner) - 1;
            const int64_t skip = (z - __shfl_sync(~0u, first, from)) * tile_rows;
            const int64_t ra = __shfl_sync(~0u, a, from), rb = __shfl_sync(~0u, b, from);
            t.row0 = (int)(ra + skip);
            t.rows = (int)min((int64_t)tile_rows, rb - ra - skip);
            t.group = g0 + from;
            return true;
        }
        before += __shfl_sync(~0u, upto, 31);
    }
    return false;
}

}  // namespace sorted
}  // namespace mse
