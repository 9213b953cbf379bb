// Rounding to 8 bits, the dispatch of routed tokens, their weighted sum, and the generic
// (CUDA-core) products that serve any size, pitch and alignment.
#include "fp8.cuh"
#include "launch.h"
#include "routed.h"

namespace mse {
namespace routed {
namespace {

// ---------------------------------------------------------------------------
// rounding to 8 bits
// ---------------------------------------------------------------------------

// eight bf16 values at `src`, a multiple of `align` bytes, of which `left` are there (fewer than one: none; the others 0).  Not by
// the read-only path: a grid begins while the kernel before it may still write what it reads after its wait.
__device__ __forceinline__ uint4 load8(const uint16_t *src, int64_t left, int align) {
    if (left >= 8 && align == 16) return *reinterpret_cast<const uint4 *>(src);
    if (left >= 8 && align == 8) {
        const uint2 lo = *reinterpret_cast<const uint2 *>(src), hi = reinterpret_cast<const uint2 *>(src)[1];
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    if (left >= 8 && align == 4) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(src);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = (2 * i < left ? src[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)src[2 * i + 1] << 16 : 0u);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint2 e4m3x8(uint4 w, const E4m3Scale &s) {
    return make_uint2(e4m3x4(w.x, w.y, s), e4m3x4(w.z, w.w, s));
}

// One block of 128 values of a row, by 16 lanes with 8 values each, 8 l .. 8 l + 7 by lane l: amax over the lanes, then this
// lane's values rounded
__device__ __forceinline__ void round_block8(uint4 w, uint32_t mask, float &a, uint2 &q) {
    uint32_t m = abs_max8(w);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(mask, m, d));
    a = floored_amax(bits_of_max2(m));
    q = e4m3x8(w, e4m3_scale(a));
}

__device__ __forceinline__ void store8(uint8_t *dst, int64_t left, bool wide, uint2 q) {
    if (wide && left >= 8) {
        *reinterpret_cast<uint2 *>(dst) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) dst[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (i % 4 * 8));
    }
}

// A block is eight lanes' with 16 values each: three exchanges for its amax, one 16-byte store a lane.  kInFlight blocks of a lane are on
// their way at once: 12288 x 7168 in 46 us (5.8 TB/s), with one 50 and with four 52 us (79 registers); 16 lanes of 8 values
// took 61 us.  2111 x 6100, rows at multiples of 8 bytes, 10.4 us (16.2 with 2-byte loads).
constexpr int kInFlight = 2;

__global__ void __launch_bounds__(256) quantise_rows_kernel(const uint16_t *x, int64_t rows, int64_t K, int64_t ldx,
                                                            int align, uint8_t *q, int64_t ldq, int wide_out,
                                                            float *scales) {
    pdl_wait();
    // (after the wait: what the next kernel reads early is complete before this kernel began)
    pdl_launch_dependents();
    const int64_t kb = (K + kBlock - 1) / kBlock, items = rows * kb;
    const int l = threadIdx.x % 8;
    const uint32_t mask = 0xFFu << (threadIdx.x & 24);
    const int64_t stride = (int64_t)gridDim.x * 32, dr = stride / kb, db = stride % kb;
    int64_t it = (int64_t)blockIdx.x * 32 + threadIdx.x / 8;
    int64_t r = it / kb, b = it % kb;   // then advanced by (dr, db): no division per block
    while (it < items) {
        uint4 lo[kInFlight], hi[kInFlight];
        int64_t rf = r, bf = b;
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int64_t k = bf * kBlock + l * 16;
            const uint16_t *src = x + rf * ldx + k;
            if (it + i * stride < items) lo[i] = load8(src, K - k, align), hi[i] = load8(src + 8, K - k - 8, align);
            rf += dr;
            bf += db;
            if (bf >= kb) { bf -= kb; ++rf; }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            if (it < items) {   // the same for the 8 lanes
                uint32_t m = __vmaxu2(abs_max8(lo[i]), abs_max8(hi[i]));
#pragma unroll
                for (int d = 4; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(mask, m, d));
                const float a = floored_amax(bits_of_max2(m));
                const E4m3Scale scale = e4m3_scale(a);
                const uint2 o = e4m3x8(lo[i], scale), o2 = e4m3x8(hi[i], scale);
                const int64_t k = b * kBlock + l * 16;
                uint8_t *dst = q + r * ldq + k;
                if (wide_out && K - k >= 16) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(o.x, o.y, o2.x, o2.y);
                } else {
                    store8(dst, K - k, false, o);
                    store8(dst + 8, K - k - 8, false, o2);
                }
                if (l == 0) scales[it] = block_scale(a);
            }
            it += stride;
            r += dr;
            b += db;
            if (b >= kb) { b -= kb; ++r; }
        }
    }
}

// One 128 x 128 block per CTA: thread (h, l) holds values 8 l .. 8 l + 7 of rows h, h + 16, .. as they were read, all eight loads on
// their way at once, until the block's amax is known.  Bound by the memory: 12288 x 7168 in 46 us, 5.8 TB/s;
// 7168 x 6144 26 us (330 and 175 with the block read twice, a value at a time).
__global__ void __launch_bounds__(256) quantise_tiles_kernel(const uint16_t *x, int64_t rows, int64_t K, int64_t ldx,
                                                             int align, uint8_t *q, int64_t ldq, int wide_out,
                                                             float *scales) {
    __shared__ uint32_t part[8];
    pdl_wait();
    const int l = threadIdx.x % 16, h = threadIdx.x / 16;
    const uint32_t kb = (uint32_t)((K + kBlock - 1) / kBlock);
    const int64_t r0 = (int64_t)(blockIdx.x / kb) * kBlock + h, k = (int64_t)(blockIdx.x % kb) * kBlock + l * 8;
    uint4 raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 16;
        raw[i] = r < rows ? load8(x + r * ldx + k, K - k, align) : make_uint4(0, 0, 0, 0);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, abs_max8(raw[i]));
    m = __reduce_max_sync(~0u, bits_of_max2(m));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, part[w]);
    const float a = floored_amax(m);
    const E4m3Scale scale = e4m3_scale(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 16;
        if (r < rows) store8(q + r * ldq + k, K - k, wide_out, e4m3x8(raw[i], scale));
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = block_scale(a);
}

// fp32 rows of the tiles of a dispatch, one warp per block of 128
__global__ void __launch_bounds__(256) quantise_f32_kernel(const float *h, const int *n_tiles, const Tile *tiles,
                                                           int64_t K, uint8_t *q, int64_t ldq, float *scales) {
    pdl_wait();
    if ((int)blockIdx.x >= *n_tiles) return;
    const Tile t = tiles[blockIdx.x];
    const int64_t kb = (K + kBlock - 1) / kBlock, items = t.rows * kb;
    const int lane = threadIdx.x % 32;
    for (int64_t it = (int64_t)blockIdx.y * 8 + threadIdx.x / 32; it < items; it += (int64_t)gridDim.y * 8) {
        const int64_t r = t.row0 + it / kb, b = it % kb;
        float v[4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = b * kBlock + i * 32 + lane;
            v[i] = k < K ? h[r * K + k] : 0.f;
            m = max(m, abs_bits(v[i]));
        }
        const float a = floored_amax(__reduce_max_sync(~0u, m)), inv = __frcp_rn(a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = b * kBlock + i * 32 + lane;
            if (k < K) q[r * ldq + k] = e4m3_of(v[i], a, inv);
        }
        if (lane == 0) scales[r * kb + b] = block_scale(a);
    }
}

// ---------------------------------------------------------------------------
// dispatch: pairs sorted by expert, their tokens in 8 bits at the sorted rows
// ---------------------------------------------------------------------------

// expert of pair i on this rank, or -1
__device__ __forceinline__ int local_expert(const DispatchParams &p, int64_t i) {
    const int64_t e = (int64_t)p.ids[i] - p.first_expert;
    return e >= 0 && e < p.E ? (int)e : -1;
}

__global__ void __launch_bounds__(kDispatchThreads) count_kernel(const DispatchParams p) {
    extern __shared__ int count_smem[];
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += kDispatchThreads) count_smem[e] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * p.chunk * p.top_k;
    const int64_t i1 = min(i0 + (int64_t)p.chunk * p.top_k, p.T * p.top_k);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kDispatchThreads) {
        const int e = local_expert(p, i);
        if (e >= 0) atomicAdd(&count_smem[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kDispatchThreads) p.hist[(int64_t)blockIdx.x * p.E + e] = count_smem[e];
}

// hist[c][e] becomes the pairs of expert e in the chunks before c; row n_chunks: in all of them.  Lane: an expert, warp: a
// 32nd of the chunks, added up first and then run through.  (Each CTA of the dispatch adding up the whole table took
// n_chunks^2: 32768 tokens with 8 of 256 experts 1112 us there, 157 now; 4096 tokens 81 and 21.)
constexpr int kScanThreads = 1024;

__global__ void __launch_bounds__(kScanThreads) scan_kernel(int *hist, int n_chunks, int E) {
    __shared__ int sums[32][33];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, e = (int)blockIdx.x * 32 + lane;
    const int per = (n_chunks + 31) / 32, c0 = min(warp * per, n_chunks), c1 = min(c0 + per, n_chunks);
    int sum = 0;
    if (e < E)
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += hist[(int64_t)c * E + e];
    sums[warp][lane] = sum;
    __syncthreads();
    if (e >= E) return;
    int run = 0;
    for (int w = 0; w < warp; ++w) run += sums[w][lane];
    for (int c = c0; c < c1; c += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < c1 ? hist[(int64_t)(c + i) * E + e] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i < c1) hist[(int64_t)(c + i) * E + e] = run;
            run += v[i];
        }
    }
    if (warp == 31) hist[(int64_t)n_chunks * E + e] = run;
}

// exclusive prefix sum of v[0 .. n) in shared memory by one warp; the total is returned
__device__ __forceinline__ int warp_prefix(int *v, int n, int lane) {
    int run = 0;
    for (int c = 0; c < n; c += 32) {
        const int mine = c + lane < n ? v[c + lane] : 0;
        int s = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(~0u, s, d);
            if (lane >= d) s += o;
        }
        if (c + lane < n) v[c + lane] = run + s - mine;
        run += __shfl_sync(~0u, s, 31);
    }
    return run;
}

// CTA (c, y): the sorted rows of token chunk c, and its k-blocks [y * per, (y + 1) * per) in 8 bits
// at those rows.  A pair's row is its expert's first row plus the pairs of that expert before it,
// counted, not drawn by atomics, so every CTA of a chunk finds the same rows.
__global__ void __launch_bounds__(kDispatchThreads) dispatch_kernel(const DispatchParams p) {
    extern __shared__ int dispatch_smem[];
    int *total = dispatch_smem, *before = total + p.E, *tile_at = before + p.E, *of_warp = tile_at + p.E;
    __shared__ int pair_row[kDispatchPairs];
    __shared__ int64_t pair_at[kDispatchPairs];   // byte offset of the row in xq, -1: none
    __shared__ int all;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t pairs = p.T * p.top_k, i0 = (int64_t)blockIdx.x * p.chunk * p.top_k;
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    const int tokens = (int)min((int64_t)p.chunk, p.T - t0), mine = tokens * p.top_k;
    for (int i = tid; i < kDispatchThreads / 32 * p.E; i += kDispatchThreads) of_warp[i] = 0;
    if (p.hist) {
        for (int e = tid; e < p.E; e += kDispatchThreads) {
            total[e] = p.hist[(int64_t)p.n_chunks * p.E + e];
            before[e] = p.hist[(int64_t)blockIdx.x * p.E + e];
        }
        __syncthreads();
    } else {
        for (int e = tid; e < p.E; e += kDispatchThreads) total[e] = before[e] = 0;
        __syncthreads();
        for (int64_t i = tid; i < pairs; i += kDispatchThreads) {
            const int e = local_expert(p, i);
            if (e >= 0) {
                atomicAdd(&total[e], 1);
                if (i < i0) atomicAdd(&before[e], 1);
            }
        }
    }
    // pair `tid` of the chunk: the pairs of its expert before it in its warp, and per warp and expert
    static_assert(kDispatchPairs <= kDispatchThreads, "one pair per thread");
    const int expert = tid < mine ? local_expert(p, i0 + tid) : -1;
    const uint32_t same = __match_any_sync(~0u, expert);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (expert >= 0 && rank == 0) of_warp[warp * p.E + expert] = __popc(same);
    __syncthreads();
    if (warp == 0) {   // each expert's first row
        const int n = warp_prefix(total, p.E, lane);
        if (lane == 0) all = n;
    }
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0) {   // writes the tiles
        for (int e = tid; e < p.E; e += kDispatchThreads)
            tile_at[e] = ((e + 1 < p.E ? total[e + 1] : all) - total[e] + p.tile_rows - 1) / p.tile_rows;
        __syncthreads();
        if (warp == 0) {
            const int n = warp_prefix(tile_at, p.E, lane);
            if (lane == 0) *p.n_tiles = n;
        }
        __syncthreads();
        for (int e = tid; e < p.E; e += kDispatchThreads) {
            const int row0 = total[e], rows = (e + 1 < p.E ? total[e + 1] : all) - row0;
            for (int k = 0; k * p.tile_rows < rows; ++k)
                p.tiles[tile_at[e] + k] = Tile{row0 + k * p.tile_rows, min(p.tile_rows, rows - k * p.tile_rows), e, 0};
        }
    }
    if (tid < mine) {
        int row = -1;
        if (expert >= 0) {
            row = total[expert] + before[expert] + rank;
            for (int w = 0; w < warp; ++w) row += of_warp[w * p.E + expert];
        }
        pair_row[tid] = row;
        pair_at[tid] = row < 0 ? -1 : (int64_t)row * p.ldq;
        if (blockIdx.y == 0) p.pos[i0 + tid] = row;
    }
    __syncthreads();
    const int64_t kb = (p.H + kBlock - 1) / kBlock;
    const int64_t per = (kb + gridDim.y - 1) / gridDim.y, b0 = blockIdx.y * per, nb = min(per, kb - b0);
    if (nb <= 0) return;
    const int l = tid % 16;
    const uint32_t mask = 0xFFFFu << (tid & 16);
    // half-warp h: tokens h, h + 16, .. of the chunk, block after block; of fewer than 16 tokens, several share one
    const int h = tid / 16, across = min(tokens, 16), stride = max(1, 16 / across);
    if (h >= across * stride) return;
    for (int t = h % across; t < tokens; t += 16) {
        const uint16_t *row = p.x + (t0 + t) * p.H;
        const int j0 = t * p.top_k;
        const int mine_row = l < p.top_k ? pair_row[j0 + l] : -1;
        auto block = [&](int b) {
            const int64_t k = (b0 + b) * kBlock + l * 8;
            return load8(row + k, p.H - k, p.align);
        };
        uint4 next = make_uint4(0, 0, 0, 0);
        int b = h / across;
        if (b < nb) next = block(b);
        for (; b < nb; b += stride) {
            const uint4 now = next;
            if (b + stride < nb) next = block(b + stride);   // while this one is rounded
            float a;
            uint2 q;
            round_block8(now, mask, a, q);
            const float s = block_scale(a);
            const int64_t k = (b0 + b) * kBlock + l * 8;
            if (k + 8 <= p.H) {
                uint8_t *dst = p.xq + k;
#pragma unroll 4
                for (int j = 0; j < p.top_k; ++j) {
                    const int64_t at = pair_at[j0 + j];
                    if (at >= 0) *reinterpret_cast<uint2 *>(dst + at) = q;
                }
            } else {
                for (int j = 0; j < p.top_k; ++j) {
                    const int64_t at = pair_at[j0 + j];
                    if (at >= 0) store8(p.xq + at + k, p.H - k, false, q);
                }
            }
            // lane l writes the scale of the token's pair l (and l + 16)
            if (mine_row >= 0) p.xs[(int64_t)mine_row * kb + b0 + b] = s;
            if (l + 16 < p.top_k && pair_row[j0 + l + 16] >= 0)
                p.xs[(int64_t)pair_row[j0 + l + 16] * kb + b0 + b] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// y[t] = shared[t] + sum_j w o
// ---------------------------------------------------------------------------
// Bound by the fp32 rows it reads: 4096 tokens of 7168 with 8 experts each, 158 us, 6.7 TB/s (187 with y stored in 2 bytes at a
// time).  Four pairs' values on their way at once: one token of 7168 and 8 experts 1.3 us less than one after the other; eight take 70
// registers, and the 4096 tokens 17 us more.
constexpr int kPairs = 4;

// WIDE: H is a multiple of 4, and y and shared begin at multiples of 8 bytes.  o's rows always begin at 16.
template <bool WIDE>
__global__ void __launch_bounds__(256) combine_kernel(const float *o, int64_t ldo, const int32_t *pos, const float *weights,
                                                      int top_k, const uint16_t *shared, uint16_t *y, int64_t T,
                                                      int64_t H) {
    pdl_wait();
    const int64_t per = (H + 3) / 4, items = T * per;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < items; it += (int64_t)gridDim.x * 256) {
        const int64_t t = it / per, c = it % per * 4;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        if (shared) {
            const uint16_t *src = shared + t * H + c;
            if constexpr (WIDE) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(src));
                acc[0] = bf16_bits_to_f32((uint16_t)v.x), acc[1] = bf16_bits_to_f32((uint16_t)(v.x >> 16));
                acc[2] = bf16_bits_to_f32((uint16_t)v.y), acc[3] = bf16_bits_to_f32((uint16_t)(v.y >> 16));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = c + i < H ? bf16_bits_to_f32(src[i]) : 0.f;
            }
        }
        // kPairs at a time: their rows' numbers, then their values, all on their way before any is added
        for (int j0 = 0; j0 < top_k; j0 += kPairs) {
            int row[kPairs];
            float w[kPairs];
            float4 v[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const bool have = j0 + j < top_k;
                row[j] = have ? pos[t * top_k + j0 + j] : -1;
                w[j] = have ? weights[t * top_k + j0 + j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (row[j] >= 0) v[j] = __ldcs(reinterpret_cast<const float4 *>(o + row[j] * ldo + c));
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (row[j] >= 0) {
                    acc[0] = fmaf(w[j], v[j].x, acc[0]);
                    acc[1] = fmaf(w[j], v[j].y, acc[1]);
                    acc[2] = fmaf(w[j], v[j].z, acc[2]);
                    acc[3] = fmaf(w[j], v[j].w, acc[3]);
                }
        }
        uint16_t *dst = y + t * H + c, r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = f32_to_bf16_bits(acc[i]);
        if constexpr (WIDE) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(r[0] | (uint32_t)r[1] << 16, r[2] | (uint32_t)r[3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < H) dst[i] = r[i];
        }
    }
}

// ---------------------------------------------------------------------------
// generic product: 16 token rows x 16 weight rows per CTA, one thread per output
// ---------------------------------------------------------------------------
template <int EPI>
__global__ void __launch_bounds__(256) block_simt_kernel(const BlockGemm g) {
    constexpr int MATS = EPI == BLOCK_SWIGLU ? 2 : 1;
    __shared__ float sx[kSimtTileRows][kBlock + 1], sw[MATS][16][kBlock + 1];
    pdl_wait();
    Tile t;
    if (g.tiles) {
        if ((int)blockIdx.x >= *g.n_tiles) return;
        t = g.tiles[blockIdx.x];
    } else {
        t.row0 = blockIdx.x * kSimtTileRows;
        t.rows = (int)min((int64_t)kSimtTileRows, g.T - t.row0);
        t.expert = 0;
    }
    const int r = threadIdx.x / 16;
    const uint8_t *w = g.wq + (int64_t)t.expert * g.w_group_rows * g.ldw;
    const float *ws = g.ws + (int64_t)t.expert * g.ws_group;
    // (one round of columns up to 1,048,560 of them: the grid's second dimension ends at 65,535)
    for (int64_t n0 = (int64_t)blockIdx.y * 16; n0 < g.N; n0 += (int64_t)gridDim.y * 16) {
        const int64_t n = n0 + threadIdx.x % 16;
        float acc[MATS] = {};
        for (int b = 0; b < g.kb; ++b) {
            for (int i = threadIdx.x; i < 16 * kBlock; i += 256) {
                const int rr = i / kBlock, kk = i % kBlock;
                const int64_t k = (int64_t)b * kBlock + kk;
                sx[rr][kk] = rr < t.rows && k < g.K ? e4m3_to_f32(g.xq[(int64_t)(t.row0 + rr) * g.ldx + k]) : 0.f;
#pragma unroll
                for (int m = 0; m < MATS; ++m)
                    sw[m][rr][kk] =
                        n0 + rr < g.N && k < g.K ? e4m3_to_f32(w[(n0 + rr + m * g.up_rows) * g.ldw + k]) : 0.f;
            }
            __syncthreads();
            if (r < t.rows && n < g.N) {
                const float xs = g.xs[(int64_t)(t.row0 + r) * g.kb + b];
#pragma unroll
                for (int m = 0; m < MATS; ++m) {
                    float d = 0.f;
                    for (int kk = 0; kk < kBlock; ++kk) d = fmaf(sx[r][kk], sw[m][threadIdx.x % 16][kk], d);
                    acc[m] = fmaf(d, xs * ws[n / kBlock * g.kb + b + m * g.up_scales], acc[m]);
                }
            }
            __syncthreads();
        }
        if (r >= t.rows || n >= g.N) continue;
        const int64_t at = (int64_t)(t.row0 + r) * g.ldo + n;
        if constexpr (EPI == BLOCK_BF16) static_cast<uint16_t *>(g.out)[at] = f32_to_bf16_bits(acc[0]);
        if constexpr (EPI == BLOCK_F32) static_cast<float *>(g.out)[at] = acc[0];
        if constexpr (EPI == BLOCK_SWIGLU) static_cast<float *>(g.out)[at] = glu(acc[0], acc[1]);
    }
}

}  // namespace

// the largest power of two, 16 at most, that divides the address of every row, and so of every eight values of it
int align_of(const uint16_t *x, int64_t ld) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | (uintptr_t)ld * 2 | 16u;
    return (int)(bits & (~bits + 1));
}

cudaError_t launch_quantise_rows(const uint16_t *x, int64_t rows, int64_t K, int64_t ldx, uint8_t *q, int64_t ldq,
                                 float *scales, int sm_count, bool pdl, cudaStream_t s) {
    const int64_t items = rows * blocks_of(K);
    const int blocks = (int)std::min<int64_t>((items + 31) / 32, (int64_t)sm_count * 8);
    const int wide_out = ldq % 16 == 0 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
    return launch_kernel(quantise_rows_kernel, dim3((unsigned)blocks), 256, 0, pdl, 1, s, x, rows, K, ldx, align_of(x, ldx), q,
                         ldq, wide_out, scales);
}

cudaError_t launch_quantise_tiles(const uint16_t *x, int64_t rows, int64_t K, int64_t ldx, uint8_t *q, int64_t ldq,
                                  float *scales, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)(blocks_of(K) * blocks_of(rows)));   // block rows one after another
    const int wide_out = ldq % 8 == 0 && (reinterpret_cast<uintptr_t>(q) & 7u) == 0;
    return launch_kernel(quantise_tiles_kernel, grid, 256, 0, pdl, 1, s, x, rows, K, ldx, align_of(x, ldx), q, ldq, wide_out,
                         scales);
}

cudaError_t launch_quantise_f32(const float *h, const int *n_tiles, const Tile *tiles, int64_t max_tiles, int64_t K,
                                uint8_t *q, int64_t ldq, float *scales, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)max_tiles, (unsigned)std::min<int64_t>((kSimtTileRows * blocks_of(K) + 7) / 8, 64));
    return launch_kernel(quantise_f32_kernel, grid, 256, 0, pdl, 1, s, h, n_tiles, tiles, K, q, ldq, scales);
}

cudaError_t launch_dispatch(const DispatchParams &p, bool pdl, cudaStream_t s) {
    if (p.hist) {
        cudaError_t e = launch_kernel(count_kernel, dim3((unsigned)p.n_chunks), kDispatchThreads, (size_t)p.E * 4, pdl, 1,
                                      s, p);
        if (e == cudaSuccess)
            e = launch_kernel(scan_kernel, dim3((unsigned)((p.E + 31) / 32)), kScanThreads, 0, pdl, 1, s, p.hist,
                              p.n_chunks, p.E);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(dispatch_kernel, dim3((unsigned)p.n_chunks, (unsigned)p.splits), kDispatchThreads,
                         (size_t)p.E * 4 * (3 + kDispatchThreads / 32), pdl, 1, s, p);
}

cudaError_t launch_combine(const float *o, int64_t ldo, const int32_t *pos, const float *weights, int top_k,
                           const uint16_t *shared, uint16_t *y, int64_t T, int64_t H, int sm_count, bool pdl,
                           cudaStream_t s) {
    const bool wide = H % 4 == 0 && ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(shared)) & 7u) == 0;
    const int64_t items = T * ((H + 3) / 4);
    const dim3 grid((unsigned)std::min<int64_t>((items + 255) / 256, (int64_t)sm_count * 16));
    return launch_kernel(wide ? combine_kernel<true> : combine_kernel<false>, grid, 256, 0, pdl, 1, s, o, ldo, pos, weights,
                         top_k, shared, y, T, H);
}

cudaError_t launch_block_simt(const BlockGemm &g, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)(g.tiles ? g.max_tiles : (g.T + kSimtTileRows - 1) / kSimtTileRows),
                    (unsigned)std::min<int64_t>((g.N + 15) / 16, 65535));
    switch (g.epi) {
        case BLOCK_BF16: return launch_kernel(block_simt_kernel<BLOCK_BF16>, grid, 256, 0, pdl, 1, s, g);
        case BLOCK_F32: return launch_kernel(block_simt_kernel<BLOCK_F32>, grid, 256, 0, pdl, 1, s, g);
        default: return launch_kernel(block_simt_kernel<BLOCK_SWIGLU>, grid, 256, 0, pdl, 1, s, g);
    }
}

}  // namespace routed
}  // namespace mse
