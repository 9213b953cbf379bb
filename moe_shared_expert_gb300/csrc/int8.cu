// Rounding of rows to 8-bit integers, and the generic (CUDA-core) product that serves any size, pitch and alignment.
#include <cuda_fp16.h>

#include <type_traits>

#include "int8_tc.cuh"
#include "launch.h"
#include "sorted.h"

namespace mse {
namespace sorted {
namespace {

// ---------------------------------------------------------------------------
// a = max(max |r|, 2^-100),  scale = a / 127,  q = rint(127 r / a);  r = x or silu(gate) up
// ---------------------------------------------------------------------------
// A row's values stay in the registers of a warp (up to 1024) or of a CTA (up to 8192) between its amax and its rounding; longer
// rows are read again.  Eight values of a thread are one load, of as many bytes as the rows' alignment lets a load have.
// Bound by memory: 8192 x 7168 in bf16 to bytes 30 us (5.8 TB/s), 64 x 7168 1.9; to fp16 32, of whose writes a part stays in L2.  (Read
// twice a value at a time it took 120 us; with a division near the middle of two integers instead of the residual step 80.)
constexpr int round_threads(int lanes) { return lanes > 256 ? lanes : 256; }

// eight values at `at` of which `left` are there (the others 0), as they lie in memory: 4 words of bf16 or 8 of fp32
template <bool F32>
__device__ __forceinline__ void load8(const void *x, int64_t at, int64_t left, int align, uint32_t (&u)[F32 ? 8 : 4]) {
    if constexpr (F32) {
        const uint32_t *p = static_cast<const uint32_t *>(x) + at;
        if (left >= 8 && align == 16) {
            const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
            u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = i < left ? p[i] : 0u;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(x) + at;
        if (left >= 8 && align == 16) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p);
            u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
        } else if (left >= 8 && align == 8) {
            const uint2 a = reinterpret_cast<const uint2 *>(p)[0], b = reinterpret_cast<const uint2 *>(p)[1];
            u[0] = a.x, u[1] = a.y, u[2] = b.x, u[3] = b.y;
        } else if (left >= 8 && align == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = (2 * i < left ? p[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)p[2 * i + 1] << 16 : 0u);
        }
    }
}
template <bool F32>
__device__ __forceinline__ void numbers(const uint32_t (&u)[F32 ? 8 : 4], float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(F32 ? u[F32 ? 2 * i : i] : u[i] << 16);
        v[2 * i + 1] = __uint_as_float(F32 ? u[F32 ? 2 * i + 1 : i] : u[i] & 0xFFFF0000u);
    }
}

// eight rounded values, as bytes or in fp16, at `at` of a row of q; the fp16 rows' pitch is a multiple of 64
template <bool HALF>
__device__ __forceinline__ void store8(void *q, int64_t at, int64_t left, bool wide, const float (&v)[8], const RowScale &s) {
    uint64_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = int8x2_of(v[2 * i], v[2 * i + 1], s);
    if constexpr (HALF) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(m[i]) : "l"(m[i]), "l"(twice(-12582912.f)));
            const __half2 p = __floats2half2_rn(__uint_as_float((uint32_t)m[i]), __uint_as_float((uint32_t)(m[i] >> 32)));
            h[i] = s.nan ? 0u : *reinterpret_cast<const uint32_t *>(&p);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(q) + at) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __byte_perm((uint32_t)m[i], (uint32_t)(m[i] >> 32), 0x0040);
        const uint32_t lo = s.nan ? 0u : __byte_perm(b[0], b[1], 0x5410), hi = s.nan ? 0u : __byte_perm(b[2], b[3], 0x5410);
        uint8_t *dst = static_cast<uint8_t *>(q) + at;
        if (wide && left >= 8) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) dst[i] = (uint8_t)((i < 4 ? lo : hi) >> (i % 4 * 8));
        }
    }
}

// LANES threads to a row (32, 256 or 512), SLOTS times eight values of each kept (0: none, rows of any length)
// What a thread keeps of eight values: bf16 as they lie in memory (half the registers, six CTAs on an SM), or 32 bits each.  BLOCKS:
// CTAs on an SM.  Rows of one load a thread have eight (silu(gate) up of 16384 x 2048 in bf16 32.6 us, 42 with four).
template <bool F32, bool GLU, bool HALF, int LANES, int SLOTS, int BLOCKS>
__global__ void __launch_bounds__(round_threads(LANES), BLOCKS) round_rows_kernel(const RoundParams p, const int align,
                                                                                       const int wide) {
    constexpr bool kWide = F32 || GLU;
    constexpr int kRows = round_threads(LANES) / LANES, kKeep = SLOTS > 0 ? SLOTS : 1;
    __shared__ uint32_t part[2][round_threads(LANES) / 32];
    pdl_wait();
    // (after the wait: what the next kernel reads early is complete before this kernel began)
    pdl_launch_dependents();
    const int64_t rows = p.last ? min((int64_t)max(*p.last, 0), p.rows) : p.rows;
    const int l = threadIdx.x % LANES;
    int turn = 0;
    for (int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES; r < rows; r += (int64_t)gridDim.x * kRows, turn ^= 1) {
        auto values = [&](int64_t k, uint32_t (&keep)[kWide ? 8 : 4]) {
            if constexpr (GLU) {
                uint32_t a[F32 ? 8 : 4], b[F32 ? 8 : 4];
                float gate[8], up[8];
                load8<F32>(p.x, r * p.ldx + k, p.K - k, align, a);
                load8<F32>(p.x, r * p.ldx + p.K + k, p.K - k, align, b);
                numbers<F32>(a, gate);
                numbers<F32>(b, up);
#pragma unroll
                for (int i = 0; i < 8; ++i) keep[i] = __float_as_uint(swiglu(gate[i], up[i]));
            } else {
                load8<F32>(p.x, r * p.ldx + k, p.K - k, align, keep);
            }
        };
        auto largest = [&](const uint32_t (&keep)[kWide ? 8 : 4], uint32_t top) {
            if constexpr (kWide) {
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, keep[j] & 0x7FFFFFFFu);
            } else {   // each half is a maximum
#pragma unroll
                for (int j = 0; j < 4; ++j) top = __vmaxu2(top, keep[j] & 0x7FFF7FFFu);
            }
            return top;
        };
        auto rounded = [&](int64_t k, const uint32_t (&keep)[kWide ? 8 : 4], const RowScale &s) {
            float v[8];
            numbers<kWide>(keep, v);
            store8<HALF>(p.q, r * p.ldq + k, p.K - k, wide, v, s);
        };
        uint32_t keep[kKeep][kWide ? 8 : 4], top = 0;
        if constexpr (SLOTS > 0) {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                const int64_t k = (int64_t)(i * LANES + l) * 8;
                if (k < p.K) values(k, keep[i]);
            }
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                if ((int64_t)(i * LANES + l) * 8 < p.K) top = largest(keep[i], top);
        } else {
            for (int64_t k = (int64_t)l * 8; k < p.K; k += LANES * 8) {
                values(k, keep[0]);
                top = largest(keep[0], top);
            }
        }
        if constexpr (!kWide) top = max(top << 16, top & 0xFFFF0000u);
        top = __reduce_max_sync(~0u, top);
        if constexpr (LANES > 32) {   // (rows in turn have buffers in turn: one barrier a row)
            if (threadIdx.x % 32 == 0) part[turn][threadIdx.x / 32] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < LANES / 32; ++w) top = max(top, part[turn][w]);
        }
        const RowScale s = row_scale(top);
        if constexpr (SLOTS > 0) {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                const int64_t k = (int64_t)(i * LANES + l) * 8;
                if (k < p.K) rounded(k, keep[i], s);
            }
        } else {
            for (int64_t k = (int64_t)l * 8; k < p.K; k += LANES * 8) {
                values(k, keep[0]);
                rounded(k, keep[0], s);
            }
        }
        if (l == 0) p.scales[r] = s.scale;
    }
}

// ---------------------------------------------------------------------------
// int8 rows to the same integers in fp16, for the tensor-core kernels
// ---------------------------------------------------------------------------
// Bound by memory: 16384 x 2048 19 us, 5.2 TB/s.  16 values a thread, two such runs on their way at once; WIDE: rows begin at
// multiples of 16 bytes (out's always do).
constexpr int kExpandRuns = 2;

template <bool WIDE>
__global__ void __launch_bounds__(256) expand_kernel(const int8_t *x, int64_t ldx, int64_t rows, int64_t K, const int32_t *last,
                                                     uint16_t *out, int64_t ldo) {
    pdl_wait();
    pdl_launch_dependents();
    if (last) rows = min((int64_t)max(*last, 0), rows);
    const uint32_t per = (uint32_t)((K + 15) / 16);   // (K below 2^17)
    const int64_t items = rows * per, stride = (int64_t)gridDim.x * 256;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += stride * kExpandRuns) {
        uint32_t w[kExpandRuns][4];
        int64_t to[kExpandRuns];
#pragma unroll
        for (int u = 0; u < kExpandRuns; ++u) {
            const int64_t i = it + u * stride;
            if (i >= items) break;
            const int64_t r = items >> 32 ? i / per : (uint32_t)i / per;
            const int64_t k = (i - r * per) * 16;
            const int8_t *src = x + r * ldx + k;
            to[u] = r * ldo + k;
            if (WIDE && k + 16 <= K) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src);
                w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (j % 4 == 0) w[u][j / 4] = 0;
                    if (k + j < K) w[u][j / 4] |= (uint32_t)(uint8_t)src[j] << (j % 4 * 8);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kExpandRuns; ++u) {
            if (it + u * stride >= items) break;
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) half_of_bytes(w[u][j], h[2 * j], h[2 * j + 1]);
            // (out's pitch is a multiple of 64 values: a run that begins inside a row is written whole)
            uint4 *dst = reinterpret_cast<uint4 *>(out + to[u]);
            dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
            dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
}

// ---------------------------------------------------------------------------
// generic product: 16 token rows x 16 weight rows per CTA, one thread per output
// ---------------------------------------------------------------------------
constexpr int kSimtRows = 16, kSimtInner = 64;

__global__ void __launch_bounds__(256) int8_simt_kernel(const Int8Gemm g) {
    // (read as words; a row is 17 of them)
    __shared__ __align__(16) int8_t sx[16][kSimtInner + 4];
    __shared__ __align__(16) int8_t sw[16][kSimtInner + 4];
    pdl_wait();
    RowTile t;
    if (!row_tile(g.offsets, g.groups, g.T, kSimtRows, blockIdx.x, t)) return;
    const int r = threadIdx.x / 16;
    const int8_t *w = g.wq + (int64_t)t.group * g.N * g.ldw;
    for (int64_t n0 = (int64_t)blockIdx.y * 16; n0 < g.N; n0 += (int64_t)gridDim.y * 16) {
        const int64_t n = n0 + threadIdx.x % 16;
        int acc = 0;
        for (int64_t k0 = 0; k0 < g.K; k0 += kSimtInner) {
            for (int i = threadIdx.x; i < 16 * kSimtInner; i += 256) {
                const int rr = i / kSimtInner, kk = i % kSimtInner;
                const int64_t k = k0 + kk;
                sx[rr][kk] = rr < t.rows && k < g.K ? g.xq[(int64_t)(t.row0 + rr) * g.ldx + k] : (int8_t)0;
                sw[rr][kk] = n0 + rr < g.N && k < g.K ? w[(n0 + rr) * g.ldw + k] : (int8_t)0;
            }
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kSimtInner; kk += 4)
                acc = __dp4a(*reinterpret_cast<const int *>(&sx[r][kk]), *reinterpret_cast<const int *>(&sw[threadIdx.x % 16][kk]), acc);
            __syncthreads();
        }
        if (r >= t.rows || n >= g.N) continue;
        const float y = (float)acc * g.xs[t.row0 + r] * g.ws[(int64_t)t.group * g.N + n];
        const int64_t at = (int64_t)(t.row0 + r) * g.N + n;
        if (g.out_f32)
            static_cast<float *>(g.out)[at] = y;
        else
            static_cast<uint16_t *>(g.out)[at] = f32_to_bf16_bits(y);
    }
}

}  // namespace

namespace {
template <bool F32, bool GLU, bool HALF>
cudaError_t round_of(const RoundParams &p, int sm_count, bool pdl, cudaStream_t s) {
    // of every eight values: the largest power of two, 16 at most, that divides the address of each
    const uintptr_t size = F32 ? 4 : 2;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)p.ldx * size | (GLU ? (uintptr_t)p.K * size : 0) | 16u;
    const int align = (int)(bits & (~bits + 1));
    const int wide = ((reinterpret_cast<uintptr_t>(p.q) | (uintptr_t)p.ldq) & 7u) == 0;
    auto with = [&](auto lanes, auto slots, auto blocks) {
        constexpr int kLanes = decltype(lanes)::value, kSlots = decltype(slots)::value, kRows = round_threads(kLanes) / kLanes;
        // (more CTAs than are resident, where a row is one load: 8192 x 7168 30 us, 33 with eight an SM)
        const dim3 grid((unsigned)std::min<int64_t>((p.rows + kRows - 1) / kRows, (int64_t)sm_count * (kSlots > 0 ? 32 : 8)));
        return launch_kernel(round_rows_kernel<F32, GLU, HALF, kLanes, kSlots, decltype(blocks)::value>, grid, round_threads(kLanes), 0,
                             pdl, 1, s, p, align, wide);
    };
    using std::integral_constant;
    constexpr bool kWide = F32 || GLU;
    if (p.K <= 256) return with(integral_constant<int, 32>(), integral_constant<int, 1>(), integral_constant<int, kWide ? 4 : 6>());
    if (p.K <= 1024) return with(integral_constant<int, 32>(), integral_constant<int, 4>(), integral_constant<int, kWide ? 4 : 6>());
    if (p.K <= 2048) return with(integral_constant<int, 256>(), integral_constant<int, 1>(), integral_constant<int, 8>());
    if constexpr (GLU) {   // (us with 256 threads a row and 512: 8192 x 4096 in bf16 40.0, 35.7; 64 x 7168 2.9, 2.5; without gate and up
                           // fp32 rows 43.7, 47.1)
        if (p.K <= 4096) return with(integral_constant<int, 512>(), integral_constant<int, 1>(), integral_constant<int, 4>());
        if (p.K <= 8192) return with(integral_constant<int, 512>(), integral_constant<int, 2>(), integral_constant<int, 3>());
    } else {
        if (p.K <= 4096) return with(integral_constant<int, 256>(), integral_constant<int, 2>(), integral_constant<int, F32 ? 4 : 6>());
        if (p.K <= 8192) return with(integral_constant<int, 256>(), integral_constant<int, 4>(), integral_constant<int, F32 ? 4 : 6>());
    }
    return with(integral_constant<int, 256>(), integral_constant<int, 0>(), integral_constant<int, kWide ? 4 : 6>());
}
}  // namespace

cudaError_t launch_int8_round(const RoundParams &p, int sm_count, bool pdl, cudaStream_t s) {
    if (p.half_out) return p.f32 ? round_of<true, false, true>(p, sm_count, pdl, s) : round_of<false, false, true>(p, sm_count, pdl, s);
    if (p.swiglu) return p.f32 ? round_of<true, true, false>(p, sm_count, pdl, s) : round_of<false, true, false>(p, sm_count, pdl, s);
    return p.f32 ? round_of<true, false, false>(p, sm_count, pdl, s) : round_of<false, false, false>(p, sm_count, pdl, s);
}

cudaError_t launch_int8_expand(const int8_t *x, int64_t ldx, int64_t rows, int64_t K, const int32_t *last, uint16_t *out,
                               int64_t ldo, int sm_count, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>((rows * ((K + 15) / 16) + 255) / 256, (int64_t)sm_count * 16));
    const bool wide = ((reinterpret_cast<uintptr_t>(x) | (uint64_t)ldx) & 15u) == 0;
    return launch_kernel(wide ? expand_kernel<true> : expand_kernel<false>, grid, 256, 0, pdl, 1, s, x, ldx, rows, K, last, out, ldo);
}

cudaError_t launch_int8_simt(const Int8Gemm &g, bool pdl, cudaStream_t s) {
    const int64_t tiles = (g.T + kSimtRows - 1) / kSimtRows + (g.offsets ? std::min<int64_t>(g.groups, g.T) : 0);
    const dim3 grid((unsigned)tiles, (unsigned)std::min<int64_t>((g.N + 15) / 16, 65535));
    return launch_kernel(int8_simt_kernel, grid, 256, 0, pdl, 1, s, g);
}

}  // namespace sorted
}  // namespace mse
