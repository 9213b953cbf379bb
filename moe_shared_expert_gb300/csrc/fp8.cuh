// Rounding to e4m3 with one scale for each block, shared by the kernels that do it.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace mse {
namespace routed {

constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100: scales stay normal numbers
constexpr float kE4m3Max = 448.f;

// |v| as an integer that orders like the number, infinities and NaN above every finite value, so
// that a maximum over it keeps a NaN
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float floored_amax(uint32_t bits) {
    return __uint_as_float(max(bits, __float_as_uint(kAmaxFloor)));   // NaN orders above and stays
}

__device__ __forceinline__ float block_scale(float a) { return __fdiv_rn(a, kE4m3Max); }

// 448 v / a for an a of floored_amax(): (448 / 512) v first, so that nothing overflows; 512 is exact.
// `inv` is 1 / a to nearest.  One residual step makes every quotient that 32 bits hold exact (q's
// error is a few units in the last place, the residual is exact, and so the step's error lies far
// below half a unit), ties of e4m3 among them; the others are nowhere near a tie when v and a are
// bf16.  Infinite v or a: NaN, like the quotient's product with the scale.  (h, which is in 32 bits, is rounded by this in the
// swap-AB kernel and by one product with 448 / a in the CTA-pair kernel: the two differ, as their sums do, where h lies in the
// last bits beside the middle of two e4m3 values.)
__device__ __forceinline__ float e4m3_ratio(float v, float a, float inv) {
    const float t = v * 0.875f, q = t * inv;
    return fmaf(fmaf(-a, q, t), inv, q) * 512.f;
}
__device__ __forceinline__ uint8_t e4m3_of(float v, float a, float inv) {
    return __nv_cvt_float_to_fp8(e4m3_ratio(v, a, inv), __NV_SATFINITE, __NV_E4M3);
}

// two values, already in e4m3's range, in 16 bits
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The same for bf16 pairs as they lie in memory, two at a time in the packed 32-bit instructions (half the instructions:
// 12288 x 7168 by rows 61 us against 68).  512 goes into 1 / a here; a / 512 and its reciprocal are normal numbers whatever a is.
struct E4m3Scale {
    uint64_t inv, minus_a;   // 512 / a and -a / 512, each twice
};
__device__ __forceinline__ uint64_t twice(float v) {
    const uint64_t u = __float_as_uint(v);
    return u | u << 32;
}
__device__ __forceinline__ E4m3Scale e4m3_scale(float a) {
    const float b = a * 0.001953125f;
    return {twice(__frcp_rn(b)), twice(-b)};
}
// two bf16 in `u`, to two e4m3
__device__ __forceinline__ uint32_t e4m3x2(uint32_t u, const E4m3Scale &s) {
    uint64_t t = (uint64_t)(u & 0xFFFF0000u) << 32 | (uint64_t)(u << 16), q, r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(t), "l"(twice(0.875f)));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(t), "l"(s.inv));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(s.minus_a), "l"(q), "l"(t));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(r), "l"(s.inv), "l"(q));
    return e4m3x2(__uint_as_float((uint32_t)q), __uint_as_float((uint32_t)(q >> 32)));
}
__device__ __forceinline__ uint32_t e4m3x4(uint32_t lo, uint32_t hi, const E4m3Scale &s) {
    return e4m3x2(lo, s) | e4m3x2(hi, s) << 16;
}

// abs_bits() of bf16 pairs: each half is a maximum
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t u) { return __vmaxu2(m, u & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t abs_max8(uint4 w) {
    return abs_max2(abs_max2(abs_max2(w.x & 0x7FFF7FFFu, w.y), w.z), w.w);
}
__device__ __forceinline__ uint32_t bits_of_max2(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }

// silu(g) u = g u / (1 + e^-g), without the care that the general exponential and quotient take of subnormal numbers:
// e^-g below 2^-126 counts as 0 and 1 / (1 + e^-g) too, for g beyond 87 either way, where the result is g u or nothing.
// Otherwise the rounding of g log2(e) makes e^-g wrong by up to 1.3 |g| 2^-24 of itself (2^-20.3 at g = -10, 2^-17.3 at
// -80), and the two approximations by a few 2^-23 more: h keeps four bits of it.  (64 of these a thread were a quarter of gate and up at K = 768; the layer of 1367 tokens with 8 of 32
// experts of 768 x 1792 takes 112 us, 140 with the general ones.)
__device__ __forceinline__ float glu(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return g * r * u;
}

// the larger of m and |v|, NaN if either is
__device__ __forceinline__ float abs_max_nan(float m, float v) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v)));
    return m;
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t q) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E4M3)));
}

}  // namespace routed
}  // namespace mse
