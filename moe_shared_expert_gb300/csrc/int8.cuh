// Rounding to 8-bit integers with one scale for each row, shared by the kernels that do it.
#pragma once
#include "common.cuh"

namespace mse {
namespace sorted {

constexpr float kInt8AmaxFloor = 7.888609052210118e-31f;   // 2^-100: scales stay normal numbers
constexpr float kLevels = 127.f;

// |v| as an integer that orders like the number, infinities and NaN above every finite value
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// A row's largest magnitude and what follows from it: 512 / a and -a / 512, each twice, for the packed 32-bit instructions.
struct RowScale {
    uint64_t inv, minus_a;
    float scale;
    bool nan;
};
__device__ __forceinline__ uint64_t twice(float v) {
    const uint64_t u = __float_as_uint(v);
    return u | u << 32;
}
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    RowScale r;
    r.nan = top >= 0x7F800000u;   // infinity or NaN: the row stands for NaN
    const float a = r.nan ? 1.f : fmaxf(__uint_as_float(top), kInt8AmaxFloor);
    const float b = a * 0.001953125f;   // and its reciprocal: normal numbers whatever a is
    r.inv = twice(__frcp_rn(b));
    r.minus_a = twice(-b);
    r.scale = r.nan ? __uint_as_float(0x7FC00000u) : __fdiv_rn(a, kLevels);
    return r;
}

// Twice rint(127 v / a), ties to even: the integers are in the low byte of each half of the result, which holds 1.5 * 2^23 more
// than they are.  127 / 512 v first, so that nothing overflows.  One residual step (q's error is a few units in the last place, the
// residual is exact, and so the step's error lies far below half a unit) makes every quotient that 32 bits hold exact, every one halfway
// between two integers among them; with v and a in bf16 no other one is anywhere near that.
__device__ __forceinline__ uint64_t int8x2_of(float lo, float hi, const RowScale &s) {
    uint64_t t = (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo), q, r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(t), "l"(twice(kLevels / 512.f)));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(t), "l"(s.inv));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(s.minus_a), "l"(q), "l"(t));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(s.inv), "l"(q));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(q), "l"(twice(12582912.f)));
    return q;
}

// silu(g) u = g / (1 + e^-g) u.  A sixteenth of 1 + e^-g goes into the reciprocal, which has no subnormal results: 1 + e^-g itself
// is above 2^126 for g below -87.3, and for those g everything would be 0.  (One product more: 16384 x 2048 in bf16 32.6 us, 31.8.)
__device__ __forceinline__ float swiglu(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, 0.0625f, 0.0625f)));
    return g * (r * 0.0625f) * u;
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
