// Rounding of rows to 8-bit integers, and the generic (CUDA-core) product that serves any size, pitch and alignment.
#include <cuda_fp16.h>

#include "int8_tc.cuh"
#include "launch.h"
#include "sorted.h"

namespace mse {
namespace sorted {
namespace {

// ---------------------------------------------------------------------------
// a = max(max |r|, 2^-100),  scale = a / 127,  q = rint(127 r / a);  r = x or silu(gate) up
// ---------------------------------------------------------------------------
constexpr int kRoundThreads = 256;

template <bool F32>
__device__ __forceinline__ float value_at(const void *x, int64_t i) {
    if constexpr (F32)
        return static_cast<const float *>(x)[i];
    else
        return bf16_bits_to_f32(static_cast<const uint16_t *>(x)[i]);
}

// one row per CTA at a time, read twice
template <bool F32, bool GLU, bool HALF>
__global__ void __launch_bounds__(kRoundThreads) round_rows_kernel(const RoundParams p) {
    __shared__ uint32_t part[kRoundThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t rows = p.last ? min((int64_t)max(*p.last, 0), p.rows) : p.rows;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        auto value = [&](int64_t k) {
            const float v = value_at<F32>(p.x, r * p.ldx + k);
            return GLU ? swiglu(v, value_at<F32>(p.x, r * p.ldx + p.K + k)) : v;
        };
        uint32_t top = 0;
        for (int64_t k = threadIdx.x; k < p.K; k += kRoundThreads) top = max(top, magnitude(value(k)));
        top = __reduce_max_sync(~0u, top);
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRoundThreads / 32; ++w) top = max(top, part[w]);
        const RowScale s = row_scale(top);
        for (int64_t k = threadIdx.x; k < p.K; k += kRoundThreads) {
            const int q = int8_of(value(k), s);
            if constexpr (HALF)
                static_cast<__half *>(p.q)[r * p.ldq + k] = __int2half_rn(q);
            else
                static_cast<int8_t *>(p.q)[r * p.ldq + k] = (int8_t)q;
        }
        if (threadIdx.x == 0) p.scales[r] = s.scale;
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// int8 rows to the same integers in fp16, for the tensor-core kernels
// ---------------------------------------------------------------------------
// 16 values a thread; WIDE: rows begin at multiples of 16 bytes (out's always do)
template <bool WIDE>
__global__ void __launch_bounds__(256) expand_kernel(const int8_t *x, int64_t ldx, int64_t rows, int64_t K, const int32_t *last,
                                                     uint16_t *out, int64_t ldo) {
    pdl_wait();
    pdl_launch_dependents();
    if (last) rows = min((int64_t)max(*last, 0), rows);
    const int64_t per = (K + 15) / 16, items = rows * per;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t r = it / per, k = (it - r * per) * 16;
        const int8_t *src = x + r * ldx + k;
        uint32_t w[4], h[8];
        if (WIDE && k + 16 <= K) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k + 4 * i + j < K) w[i] |= (uint32_t)(uint8_t)src[4 * i + j] << (8 * j);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) half_of_bytes(w[i], h[2 * i], h[2 * i + 1]);
        // (out's pitch is a multiple of 64 values: a run that begins inside a row is written whole)
        uint4 *dst = reinterpret_cast<uint4 *>(out + r * ldo + k);
        dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
        dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
    }
}

// ---------------------------------------------------------------------------
// generic product: 16 token rows x 16 weight rows per CTA, one thread per output
// ---------------------------------------------------------------------------
constexpr int kSimtRows = 16, kSimtInner = 64;

__global__ void __launch_bounds__(256) int8_simt_kernel(const Int8Gemm g) {
    __shared__ int8_t sx[16][kSimtInner + 4], sw[16][kSimtInner + 4];
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

cudaError_t launch_int8_round(const RoundParams &p, int sm_count, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>(p.rows, (int64_t)sm_count * 8));
    auto with = [&](auto f32, auto glu) {
        if (p.half_out) return launch_kernel(round_rows_kernel<decltype(f32)::value, decltype(glu)::value, true>, grid, kRoundThreads, 0, pdl, 1, s, p);
        return launch_kernel(round_rows_kernel<decltype(f32)::value, decltype(glu)::value, false>, grid, kRoundThreads, 0, pdl, 1, s, p);
    };
    if (p.f32) return p.swiglu ? with(std::true_type(), std::true_type()) : with(std::true_type(), std::false_type());
    return p.swiglu ? with(std::false_type(), std::true_type()) : with(std::false_type(), std::false_type());
}

cudaError_t launch_int8_expand(const int8_t *x, int64_t ldx, int64_t rows, int64_t K, const int32_t *last, uint16_t *out,
                               int64_t ldo, int sm_count, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>((rows * ((K + 15) / 16) + 255) / 256, (int64_t)sm_count * 8));
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
