// Tokens sorted by expert and back with weights, and the gradients of both ways.
//
// All of it moves rows: what bounds each kernel is the memory.  Nothing is drawn by atomics: a pair's place is counted, and
// every sum has one order.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "sorted.h"

namespace mse {
namespace sorted {
namespace {

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------

// expert of pair i on this rank, or -1
__device__ __forceinline__ int local_expert(const SortParams &p, int64_t i) {
    const int64_t e = (int64_t)p.ids[i] - p.first_expert;
    return e >= 0 && e < p.E ? (int)e : -1;
}

// hist[c][e] = pairs of expert e in chunk c
__global__ void __launch_bounds__(kSortThreads) count_pairs_kernel(const SortParams p) {
    extern __shared__ int count_smem[];
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) count_smem[e] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * p.chunk * p.top_k, i1 = min(i0 + (int64_t)p.chunk * p.top_k, p.T * p.top_k);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
        const int e = local_expert(p, i);
        if (e >= 0) atomicAdd(&count_smem[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) p.hist[(int64_t)blockIdx.x * p.E + e] = count_smem[e];
}

// hist[c][e] becomes the pairs of expert e in the chunks before c; row n_chunks: in all of them.  Lane: an expert, warp: a 32nd of
// the chunks, added up first and then run through.
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) scan_pairs_kernel(int *hist, int n_chunks, int E) {
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
    for (int c = c0; c < c1; ++c) {
        const int mine = hist[(int64_t)c * E + e];
        hist[(int64_t)c * E + e] = run;
        run += mine;
    }
    if (warp == 31) hist[(int64_t)n_chunks * E + e] = run;
}

// Both in one launch, by a cluster: CTA r has the chunks [r per, (r + 1) per), whose counts stay in its shared memory until it
// knows the pairs that the CTAs before it found.
constexpr int kCountCluster = 8, kCountThreads = 1024;
constexpr int kCountBytes = 160 * 1024;

__global__ void __launch_bounds__(kCountThreads) count_scan_kernel(const SortParams p, const int per) {
    extern __shared__ int cluster_smem[];
    int *counts = cluster_smem, *total = counts + per * p.E, *base = total + p.E;   // [per x E], [E], [E]
    const int tid = threadIdx.x, rank = (int)cluster_ctarank();
    pdl_wait();
    pdl_launch_dependents();
    for (int i = tid; i < per * p.E; i += kCountThreads) counts[i] = 0;
    __syncthreads();
    const int c0 = min(rank * per, p.n_chunks), c1 = min(c0 + per, p.n_chunks), pairs = p.chunk * p.top_k;
    const int64_t i0 = (int64_t)c0 * pairs;
    const int n = (int)(min((int64_t)c1 * pairs, p.T * p.top_k) - i0);
    for (int i = tid; i < n; i += kCountThreads) {
        const int e = local_expert(p, i0 + i);
        if (e >= 0) atomicAdd(&counts[i / pairs * p.E + e], 1);
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += kCountThreads) {
        int run = 0;
        for (int c = 0; c < c1 - c0; ++c) {
            const int mine = counts[c * p.E + e];
            counts[c * p.E + e] = run;
            run += mine;
        }
        total[e] = run;
    }
    cluster_sync();
    for (int e = tid; e < p.E; e += kCountThreads) {
        int before = 0, all = 0;
        for (int r = 0; r < kCountCluster; ++r) {
            int v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(total + e), (uint32_t)r)) : "memory");
            if (r < rank) before += v;
            all += v;
        }
        base[e] = before;
        if (rank == 0) p.hist[(int64_t)p.n_chunks * p.E + e] = all;
    }
    cluster_sync();   // (and nobody is over while others read its totals)
    for (int i = tid; i < (c1 - c0) * p.E; i += kCountThreads) p.hist[(int64_t)c0 * p.E + i] = base[i % p.E] + counts[i];
}

// exclusive prefix sums of v[0 .. n) in shared memory by one warp; the total is returned
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

// CTA (c, y): the places of chunk c's pairs, counted by every CTA of the chunk alike, and the y-th share of its rows' copies.
// A pair's place is its expert's first row, the expert's pairs in the chunks before, and those before it in the chunk.
// Bound by memory, most of it writes: 8192 tokens of 7168 bytes with 8 of 128 experts, 64 of them here, 51 us with the kernels that
// count (5.4 TB/s; this one alone 44); 4096 tokens of 7168 in bf16 with 8 of 32 experts 89; one token 3.1.  Rows of an odd number of
// bytes go byte by byte: 4000 tokens of 4099 bytes, 6 rows each, 39 us, of 4100 28.
template <typename W, int WORDS>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p) {
    extern __shared__ int sort_smem[];
    int *total = sort_smem, *before = total + p.E, *of_warp = before + p.E;   // of_warp: [warps x E]
    __shared__ int pair_row[kSortThreads];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (!p.hist) pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk, i0 = t0 * p.top_k;
    const int tokens = (int)min((int64_t)p.chunk, p.T - t0), mine = tokens * p.top_k;
    // The rows go by segments of kWords words a lane: (token, segment) by (token), warps of all the chunk's CTAs in turn; the next
    // one's words are on their way while one's are stored, and the first one's while places are counted.  (Behind the kernels that
    // count, which began after everything before the call was complete, x may be read before the wait.)
    constexpr int kWords = WORDS;
    const int64_t words = p.row_bytes / (int)sizeof(W);
    const int segs = (int)((words + 32 * kWords - 1) / (32 * kWords));
    const int64_t items = (int64_t)tokens * segs, stride = (int64_t)p.splits * (kSortThreads / 32);
    auto fetch = [&](int64_t it, W (&v)[kWords]) {
        const int t = (int)((uint32_t)it / (uint32_t)segs);
        const int64_t at = (it - (int64_t)t * segs) * (32 * kWords) + lane;
        const W *src = reinterpret_cast<const W *>(p.x + (t0 + t) * p.ldx) + at;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (at + 32 * i < words) v[i] = src[32 * i];
    };
    int64_t it = (int64_t)blockIdx.y * (kSortThreads / 32) + warp;
    W next[kWords];
    if (it < items) fetch(it, next);
    if (p.hist) pdl_wait();
    for (int i = tid; i < kSortThreads / 32 * p.E; i += kSortThreads) of_warp[i] = 0;
    if (p.hist) {
        for (int e = tid; e < p.E; e += kSortThreads) {
            total[e] = p.hist[(int64_t)p.n_chunks * p.E + e];
            before[e] = p.hist[(int64_t)blockIdx.x * p.E + e];
        }
        __syncthreads();
    } else {
        for (int e = tid; e < p.E; e += kSortThreads) total[e] = before[e] = 0;
        __syncthreads();
        for (int64_t i = tid; i < p.T * p.top_k; i += kSortThreads) {
            const int e = local_expert(p, i);
            if (e >= 0) {
                atomicAdd(&total[e], 1);
                if (i < i0) atomicAdd(&before[e], 1);
            }
        }
    }
    // pair `tid` of the chunk: the pairs of its expert before it in its warp, and the warp's pairs of the expert
    const int expert = tid < mine ? local_expert(p, i0 + tid) : -1;
    const uint32_t same = __match_any_sync(~0u, expert);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (expert >= 0 && rank == 0) of_warp[warp * p.E + expert] = __popc(same);
    __syncthreads();
    if (warp == 0) {   // the experts' first rows
        const int all = warp_prefix(total, p.E, lane);
        __syncwarp();
        if (blockIdx.x == 0 && blockIdx.y == 0) {
            for (int e = lane; e < p.E; e += 32) p.offsets[e] = total[e];
            if (lane == 0) p.offsets[p.E] = all;
        }
    }
    __syncthreads();
    if (tid < mine) {
        int row = -1;
        if (expert >= 0) {
            row = total[expert] + before[expert] + rank;
            for (int w = 0; w < warp; ++w) row += of_warp[w * p.E + expert];
        }
        pair_row[tid] = row;
        if (blockIdx.y == 0) {
            p.place[i0 + tid] = row;
            if (p.scales && row >= 0) p.row_scales[row] = p.scales[t0 + tid / p.top_k];
        }
    }
    __syncthreads();
    for (; it < items; it += stride) {
        W v[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = next[i];
        if (it + stride < items) fetch(it + stride, next);
        const int t = (int)((uint32_t)it / (uint32_t)segs);
        const int64_t at = (it - (int64_t)t * segs) * (32 * kWords) + lane;
        for (int j = 0; j < p.top_k; ++j) {
            const int row = pair_row[t * p.top_k + j];
            if (row < 0) continue;
            W *dst = reinterpret_cast<W *>(p.rows + row * p.ldr) + at;
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                if (at + 32 * i < words) dst[32 * i] = v[i];
        }
    }
}

// ---------------------------------------------------------------------------
// values of 2 and 4 bytes, V at a time, in 32 bits
// ---------------------------------------------------------------------------
__device__ __forceinline__ float value_of(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float value_of(float v) { return v; }
__device__ __forceinline__ void put(uint16_t &o, float v) { o = f32_to_bf16_bits(v); }
__device__ __forceinline__ void put(float &o, float v) { o = v; }

// Words of U values, as many as the alignment of every tensor lets an access have.  A thread has one word of four or eight at a time;
// of rows that allow fewer, a warp has kSpan neighbouring values, a lane eight of them in words at steps of 32 (4000 tokens of 4099 in
// bf16, 6 rows each: 82 us and 101 back, 191 and 183 with one value a thread; of 4098, words of two, 61 and 122; of 4096 50 and 72).
constexpr int kSpan = 256;

template <typename T, int U>
struct alignas(U * sizeof(T) > 16 ? 16 : U * sizeof(T)) Word {
    T v[U];
};
// the lane's values of p[0 .. left); what lies behind it is read from the front instead, so that no load waits for a branch
template <typename T, int U>
struct Span {
    Word<T, U> w[8 / U];
    __device__ __forceinline__ void load(const T *p, int64_t left, int lane) {
#pragma unroll
        for (int i = 0; i < 8 / U; ++i) {
            const int at = (i * 32 + lane) * U;
            w[i] = *reinterpret_cast<const Word<T, U> *>(p + (at < left ? at : 0));
        }
    }
    __device__ __forceinline__ void clear_behind(int64_t left, int lane) {
#pragma unroll
        for (int i = 0; i < 8 / U; ++i)
#pragma unroll
            for (int j = 0; j < U; ++j)
                if ((i * 32 + lane) * U >= left) w[i].v[j] = T(0);
    }
    __device__ __forceinline__ void store(T *p, int64_t left, int lane, const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8 / U; ++i) {
            const int at = (i * 32 + lane) * U;
#pragma unroll
            for (int j = 0; j < U; ++j) put(w[i].v[j], f[i * U + j]);
            if (at < left) *reinterpret_cast<Word<T, U> *>(p + at) = w[i];
        }
    }
    __device__ __forceinline__ float at(int i) const { return value_of(w[i / U].v[i % U]); }
};

// ---------------------------------------------------------------------------
// y[t] = base[t] + sum_j w[t, j] rows[place[t, j]], ascending j
// ---------------------------------------------------------------------------
// Bound by memory: 4096 tokens of 7168 in bf16 with 8 rows each on top of base 90 us, 6.2 TB/s.
constexpr int kPairs = 4;   // rows of a token on their way at once

// What a thread has of a row at a time, from `at` values on: one word, or a lane's part of a span.
template <typename T, int U>
struct Single {
    Word<T, U> w;
    __device__ __forceinline__ void load(const T *p, int64_t, int) { w = *reinterpret_cast<const Word<T, U> *>(p); }
    __device__ __forceinline__ void store(T *p, int64_t, int, const float (&f)[U]) {
#pragma unroll
        for (int j = 0; j < U; ++j) put(w.v[j], f[j]);
        *reinterpret_cast<Word<T, U> *>(p) = w;
    }
    __device__ __forceinline__ float at(int i) const { return value_of(w.v[i]); }
};

template <typename R, typename Y, int U>
__global__ void __launch_bounds__(256) unsort_kernel(const UnsortParams p) {
    constexpr bool kSingle = U >= 4;
    constexpr int kValues = kSingle ? U : 8;
    using In = typename std::conditional<kSingle, Single<R, U>, Span<R, U>>::type;
    using Out = typename std::conditional<kSingle, Single<Y, U>, Span<Y, U>>::type;
    pdl_wait();
    const R *rows = static_cast<const R *>(p.rows);
    const int lane = threadIdx.x % 32;
    // items of a thread, or of a warp
    const uint32_t per = (uint32_t)(kSingle ? p.H / U : (p.H + kSpan - 1) / kSpan);
    const int64_t items = p.T * per, stride = (int64_t)gridDim.x * (kSingle ? 256 : 8);
    for (int64_t it = kSingle ? (int64_t)blockIdx.x * 256 + threadIdx.x : (int64_t)blockIdx.x * 8 + threadIdx.x / 32; it < items;
         it += stride) {
        const int64_t t = items >> 32 ? it / per : (uint32_t)it / per, c = (it - t * per) * (kSingle ? U : kSpan), left = p.H - c;
        float acc[kValues];
        if (p.base) {
            Out b;
            b.load(static_cast<const Y *>(p.base) + t * p.H + c, left, lane);
#pragma unroll
            for (int i = 0; i < kValues; ++i) acc[i] = b.at(i);
        } else {
#pragma unroll
            for (int i = 0; i < kValues; ++i) acc[i] = 0.f;
        }
        for (int j0 = 0; j0 < p.top_k; j0 += kPairs) {
            int64_t row[kPairs];
            float w[kPairs];
            In v[kPairs];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const bool have = j0 + j < p.top_k;
                row[j] = have ? p.place[t * p.top_k + j0 + j] : -1;
                w[j] = have && p.weights ? p.weights[t * p.top_k + j0 + j] : 1.f;
                if (row[j] >= p.n_rows) row[j] = -1;
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (row[j] >= 0) v[j].load(rows + row[j] * p.ldr + c, left, lane);
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (row[j] >= 0)
#pragma unroll
                    for (int i = 0; i < kValues; ++i) acc[i] = fmaf(w[j], v[j].at(i), acc[i]);
        }
        Out o;
        o.store(static_cast<Y *>(p.y) + t * p.H + c, left, lane, acc);
    }
}

// ---------------------------------------------------------------------------
// drows[place[t, j]] = w[t, j] dy[t],  dweights[t, j] = <rows[place[t, j]], dy[t]>
// ---------------------------------------------------------------------------
// A CTA has one token at a time, kPairs of its pairs at once: of kManyThreads threads, or where there are too few tokens to fill the
// SMs of kFewThreads, which take fewer steps one after another along a row.  Bound by memory: 4096 tokens of 7168 in bf16 with 8 rows
// each 147 us, 6.5 TB/s.
constexpr int kManyThreads = 128, kFewThreads = 512;

template <typename D, typename R, int U, int THREADS>
__global__ void __launch_bounds__(THREADS) unsort_backward_kernel(const UnsortBackwardParams p) {
    __shared__ float part[THREADS / 32][kPairs];
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const D *dy = static_cast<const D *>(p.dy);
    const R *rows = static_cast<const R *>(p.rows);
    R *drows = static_cast<R *>(p.drows);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        for (int j0 = 0; j0 < p.top_k; j0 += kPairs) {
            int64_t row[kPairs];
            float w[kPairs], dot[kPairs];
            bool any = false;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const bool have = j0 + j < p.top_k;
                row[j] = have ? p.place[t * p.top_k + j0 + j] : -1;
                w[j] = have && p.weights ? p.weights[t * p.top_k + j0 + j] : 1.f;
                if (row[j] >= p.n_rows) row[j] = -1;
                any |= row[j] >= 0;
                dot[j] = 0.f;
            }
            if constexpr (U >= 4) {   // one word a lane
                if (any)
                    for (int64_t c = (int64_t)threadIdx.x * U; c < p.H; c += THREADS * U) {
                        const Word<D, U> d = *reinterpret_cast<const Word<D, U> *>(dy + t * p.H + c);
                        Word<R, U> v[kPairs];
                        if (p.dweights)
    #pragma unroll
                            for (int j = 0; j < kPairs; ++j)
                                if (row[j] >= 0) v[j] = *reinterpret_cast<const Word<R, U> *>(rows + row[j] * p.ldr + c);
    #pragma unroll
                        for (int j = 0; j < kPairs; ++j)
                            if (row[j] >= 0) {
                                Word<R, U> o;
    #pragma unroll
                                for (int i = 0; i < U; ++i) {
                                    const float g = value_of(d.v[i]);
                                    if (p.dweights) dot[j] = fmaf(value_of(v[j].v[i]), g, dot[j]);
                                    put(o.v[i], w[j] * g);
                                }
                                *reinterpret_cast<Word<R, U> *>(drows + row[j] * p.ldd + c) = o;
                            }
                    }
            } else {
                auto span = [&](int64_t c, auto whole) {
                    const int64_t left = decltype(whole)::value ? kSpan : p.H - c;
                    Span<D, U> d;
                    d.load(dy + t * p.H + c, left, lane);
                    Span<R, U> v[kPairs];
                    if (p.dweights)
    #pragma unroll
                        for (int j = 0; j < kPairs; ++j)
                            if (row[j] >= 0) v[j].load(rows + row[j] * p.ldr + c, left, lane);
                    if constexpr (!decltype(whole)::value) {
                        d.clear_behind(left, lane);
    #pragma unroll
                        for (int j = 0; j < kPairs; ++j) v[j].clear_behind(left, lane);
                    }
    #pragma unroll
                    for (int j = 0; j < kPairs; ++j)
                        if (row[j] >= 0) {
                            float o[8];
    #pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float g = d.at(i);
                                if (p.dweights) dot[j] = fmaf(v[j].at(i), g, dot[j]);
                                o[i] = w[j] * g;
                            }
                            v[j].store(drows + row[j] * p.ldd + c, left, lane, o);
                        }
                };
                if (any) {
                    int64_t c = (int64_t)warp * kSpan;
                    for (; c + kSpan <= p.H; c += THREADS / 32 * kSpan) span(c, std::true_type());
                    if (c < p.H) span(c, std::false_type());
                }
            }
            if (!p.dweights) continue;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(~0u, dot[j], d);
                if (lane == 0) part[warp][j] = dot[j];
            }
            __syncthreads();
            if (warp < kPairs && j0 + warp < p.top_k) {   // a pair's sum by a warp
                constexpr int kParts = THREADS / 32;
                float sum = lane < kParts ? part[lane][warp] : 0.f;
#pragma unroll
                for (int d = kParts / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
                if (lane == 0) p.dweights[t * p.top_k + j0 + warp] = sum;
            }
            __syncthreads();
        }
    }
}

// the most values of a row, of 8, 4, 2 and 1, that one access of every tensor may take
struct Width {
    int64_t values = 0;
    int limit = 8;
    void tensor(const void *base, int64_t pitch, int size) {
        if (!base) return;
        values |= pitch;
        while (limit > 1 && (reinterpret_cast<uintptr_t>(base) % (uintptr_t)std::min(limit * size, 16)) != 0) limit /= 2;
    }
    int width() const {
        int v = limit;
        while (v > 1 && values % v != 0) v /= 2;
        return v;
    }
};

}  // namespace

// Up to this many pairs one cluster counts them.  (us of a sort with two kernels and with the cluster: 16,384 pairs of 2048 fp32 to 16 of
// 64 experts 15.0, 13.9; 8192 pairs of 2048 bf16 14.4, 12.8; 32,768 of 7168 bf16 90.4, 89.4; 65,536 of 7168 bytes 53.4, 54.6; 131,072 of
// 512 bf16 32.9, 38.7.)
constexpr int64_t kClusterPairs = 32768;

cudaError_t launch_sort(const SortParams &p, bool pdl, cudaStream_t s) {
    const int per = (p.n_chunks + kCountCluster - 1) / kCountCluster;
    const int64_t bytes = (int64_t)(per + 2) * p.E * 4;
    if (p.hist && p.T * p.top_k <= kClusterPairs && bytes <= kCountBytes) {
        static std::atomic<uint64_t> done;   // bit per device
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && !(done.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
            e = cudaFuncSetAttribute(count_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCountBytes);
            if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_acq_rel);
        }
        if (e == cudaSuccess)
            e = launch_kernel(count_scan_kernel, dim3(kCountCluster), kCountThreads, (size_t)bytes, pdl, kCountCluster, s, p, per);
        if (e != cudaSuccess) return e;
    } else if (p.hist) {
        cudaError_t e = launch_kernel(count_pairs_kernel, dim3((unsigned)p.n_chunks), kSortThreads, (size_t)p.E * 4, pdl, 1, s, p);
        if (e == cudaSuccess)
            e = launch_kernel(scan_pairs_kernel, dim3((unsigned)((p.E + 31) / 32)), kScanThreads, 0, pdl, 1, s, p.hist,
                              p.n_chunks, p.E);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)p.n_chunks, (unsigned)p.splits);
    const size_t smem = (size_t)p.E * 4 * (2 + kSortThreads / 32);
    switch (p.unit) {
        case 16:
            if (p.few) return launch_kernel(sort_kernel<uint4, 1>, grid, kSortThreads, smem, pdl, 1, s, p);
            return launch_kernel(sort_kernel<uint4, 4>, grid, kSortThreads, smem, pdl, 1, s, p);
        case 8: return launch_kernel(sort_kernel<uint2, 4>, grid, kSortThreads, smem, pdl, 1, s, p);
        case 4: return launch_kernel(sort_kernel<uint32_t, 4>, grid, kSortThreads, smem, pdl, 1, s, p);
        case 2: return launch_kernel(sort_kernel<uint16_t, 8>, grid, kSortThreads, smem, pdl, 1, s, p);
        default: return launch_kernel(sort_kernel<uint8_t, 16>, grid, kSortThreads, smem, pdl, 1, s, p);
    }
}

namespace {
template <typename R, typename Y>
cudaError_t unsort_of(const UnsortParams &p, int v, dim3 grid, bool pdl, cudaStream_t s) {
    switch (v) {
        case 8: return launch_kernel(unsort_kernel<R, Y, 8>, grid, 256, 0, pdl, 1, s, p);
        case 4: return launch_kernel(unsort_kernel<R, Y, 4>, grid, 256, 0, pdl, 1, s, p);
        case 2: return launch_kernel(unsort_kernel<R, Y, 2>, grid, 256, 0, pdl, 1, s, p);
        default: return launch_kernel(unsort_kernel<R, Y, 1>, grid, 256, 0, pdl, 1, s, p);
    }
}
template <typename D, typename R, int THREADS>
cudaError_t backward_by(const UnsortBackwardParams &p, int v, dim3 grid, bool pdl, cudaStream_t s) {
    switch (v) {
        case 8: return launch_kernel(unsort_backward_kernel<D, R, 8, THREADS>, grid, THREADS, 0, pdl, 1, s, p);
        case 4: return launch_kernel(unsort_backward_kernel<D, R, 4, THREADS>, grid, THREADS, 0, pdl, 1, s, p);
        case 2: return launch_kernel(unsort_backward_kernel<D, R, 2, THREADS>, grid, THREADS, 0, pdl, 1, s, p);
        default: return launch_kernel(unsort_backward_kernel<D, R, 1, THREADS>, grid, THREADS, 0, pdl, 1, s, p);
    }
}
template <typename D, typename R>
cudaError_t backward_of(const UnsortBackwardParams &p, int v, int sm_count, bool pdl, cudaStream_t s) {
    const dim3 grid((unsigned)std::min<int64_t>(p.T, (int64_t)sm_count * 16));
    return p.T < sm_count * 4 ? backward_by<D, R, kFewThreads>(p, v, grid, pdl, s) : backward_by<D, R, kManyThreads>(p, v, grid, pdl, s);
}
}  // namespace

cudaError_t launch_unsort(const UnsortParams &p, int sm_count, bool pdl, cudaStream_t s) {
    Width w;
    w.tensor(p.rows, p.ldr, p.rows_f32 ? 4 : 2);
    w.tensor(p.base, p.H, p.y_f32 ? 4 : 2);
    w.tensor(p.y, p.H, p.y_f32 ? 4 : 2);
    const int v = w.width();
    const int64_t ctas = v >= 4 ? (p.T * (p.H / v) + 255) / 256 : (p.T * ((p.H + kSpan - 1) / kSpan) + 7) / 8;
    const dim3 grid((unsigned)std::min<int64_t>(ctas, (int64_t)sm_count * 16));
    if (p.rows_f32)
        return p.y_f32 ? unsort_of<float, float>(p, v, grid, pdl, s) : unsort_of<float, uint16_t>(p, v, grid, pdl, s);
    return p.y_f32 ? unsort_of<uint16_t, float>(p, v, grid, pdl, s) : unsort_of<uint16_t, uint16_t>(p, v, grid, pdl, s);
}

cudaError_t launch_unsort_backward(const UnsortBackwardParams &p, int sm_count, bool pdl, cudaStream_t s) {
    Width w;
    w.tensor(p.dy, p.H, p.dy_f32 ? 4 : 2);
    w.tensor(p.rows, p.ldr, p.rows_f32 ? 4 : 2);
    w.tensor(p.drows, p.ldd, p.rows_f32 ? 4 : 2);
    const int v = w.width();
    if (p.dy_f32)
        return p.rows_f32 ? backward_of<float, float>(p, v, sm_count, pdl, s) : backward_of<float, uint16_t>(p, v, sm_count, pdl, s);
    return p.rows_f32 ? backward_of<uint16_t, float>(p, v, sm_count, pdl, s) : backward_of<uint16_t, uint16_t>(p, v, sm_count, pdl, s);
}

}  // namespace sorted
}  // namespace mse
