// Product in 8-bit integers for few token rows: weights fill the 128-row side of the MMA, up to 64 tokens are its columns.
//
// A CTA owns one 128-row weight tile and one token tile; the k-blocks may be split over a cluster, whose CTAs exchange their
// integer sums through distributed shared memory and each finish a slice of the token columns.
//
// Warp 0 loads (TMA), warp 1 issues MMAs.  Warps 2-5 and 6-9 convert the weights of every other k-block each (int8_tc.cuh), and each
// adds one half of the token columns when a chunk of k-blocks ends.
//
// Bound by memory and the launch with few tokens: 16 x 12288 x 7168 20.6 us with the kernel before it (memory alone 13; without
// conversions and MMAs 19.3), 16 x 2112 x 7168 9.9 in five parts.  With 64 tokens by the conversion and the hand-over of stages and
// slots: 64 x 12288 x 7168 24.0; 160 x 12288 x 7168 38, without conversions 31, with no tokens loaded still 38.  Two CTAs on an SM
// hide each other's hand-overs; one group of converting warps instead of two takes 64 x 2112 x 7168 from 12.4 to 16.2 us, stages of
// their own for weights and tokens 1 us more everywhere.
#include <atomic>

#include "device.h"
#include "int8_tc.cuh"
#include "launch.h"

namespace mse {
namespace sorted {
namespace {

constexpr int kMaxStages = 10;
constexpr int kColsThreads = 32 * 10;

constexpr int pow2_at_least(int v) {
    int p = 32;
    while (p < v) p <<= 1;
    return p;
}

struct ColsCtrl {
    uint64_t full[kMaxStages], empty[kMaxStages], afull[4], aempty[4], dfull[2], dempty[2], drain;
    uint32_t tmem_base;
    int abort_flag;
};

template <int BN_>
struct Cols {
    static constexpr int BN = BN_;
    static constexpr int CTAS = 2;                                       // resident per SM (the ring may take a whole SM)
    static constexpr int NA = 3;                                         // k-blocks of weights in TMEM
    static constexpr int ND = BN == 64 ? 1 : 2;                          // chunks of sums there
    static constexpr int CPT = BN / 2;                                   // token columns a thread adds
    static constexpr int TMEM = pow2_at_least(ND * BN + NA * (int)kATmem);
    static_assert(CTAS * TMEM <= 512, "TMEM");
    static constexpr uint32_t TOKENS = BN * kInner * 2;                  // two tiles of 64 k
    static constexpr uint32_t STAGE = kWeightTile + TOKENS;
    static constexpr uint32_t FIXED = 1024 + sizeof(ColsCtrl) + 64;
    static constexpr int fit(uint32_t budget) {
        const int n = (int)((budget - FIXED) / STAGE);
        return n < kMaxStages ? n : kMaxStages;
    }
    // stages of the ring with two CTAs on an SM, or one
    static constexpr int PART = fit(113 * 1024), WHOLE = fit(227 * 1024);
    static_assert(NA <= PART, "the order of waits before a conversion");
    // the exchange of a split tile uses the ring: at most BN / 4 + 7 groups of four columns
    static_assert((BN / 4 + 7) * 2048 <= PART * STAGE, "exchange");
};

template <typename C>
__global__ void __launch_bounds__(kColsThreads, C::CTAS)
    int8_cols_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Int8Gemm g,
                     const int kb_total, const int stream_weights, const int S) {
    constexpr int BN = C::BN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *ring = smem_raw + (base - raw);
    ColsCtrl *ctl = reinterpret_cast<ColsCtrl *>(ring + (size_t)S * C::STAGE);
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int part = blockIdx.x, parts = gridDim.x, m = blockIdx.z;
    const int kb0 = (int)((int64_t)kb_total * part / parts), n = (int)((int64_t)kb_total * (part + 1) / parts) - kb0;
    volatile int *abort_flag = &ctl->abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < C::NA; ++a) {
            mbar_init(smem_u32(&ctl->afull[a]), 4);
            mbar_init(smem_u32(&ctl->aempty[a]), 1);
        }
        for (int d = 0; d < C::ND; ++d) {
            mbar_init(smem_u32(&ctl->dfull[d]), 1);
            mbar_init(smem_u32(&ctl->dempty[d]), 8);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl->tmem_base), C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(~0u, ctl->tmem_base, 0), tmem_a = tmem_base + C::ND * BN;
    // The kernel before this one, of the same call, let this one start after its own wait: weights and offsets are complete,
    // and only the tokens are that kernel's.
    RowTile t;
    const bool active = row_tile(g.offsets, g.groups, g.T, BN, blockIdx.y, t);
    if (!active || warp >= 2) pdl_wait();   // (a CTA without a tile too: the grid may not be over before the kernel before it)

    int issued = 0;
    if (active && warp == 0) {
        const bool el = elected();
        const int w_row = t.group * (int)g.N + m * 128;
        const uint64_t pol_w = stream_weights ? l2_policy_evict_first() : l2_policy_evict_last();
        const uint64_t pol_x = l2_policy_evict_last();
        auto weights = [&](int s, int kb) {
            const uint32_t bar = smem_u32(&ctl->full[s]);
            mbar_arrive_expect_tx(bar, C::STAGE);
            tma_load_2d(base + s * C::STAGE, &tmW, bar, kb * kInner, w_row, pol_w);
        };
        auto tokens = [&](int s, int kb) {
            const uint32_t bar = smem_u32(&ctl->full[s]), dst = base + s * C::STAGE + kWeightTile;
            tma_load_2d(dst, &tmX, bar, kb * 2 * kInner, t.row0, pol_x);   // coordinates in bytes
            tma_load_2d(dst + C::TOKENS / 2, &tmX, bar, kb * 2 * kInner + kInner, t.row0, pol_x);
        };
        const int pre = min(S, n);
        for (int i = 0; i < pre; ++i)
            if (el) weights(i, kb0 + i);
        pdl_wait();
        for (int i = 0; i < pre; ++i)
            if (el) tokens(i, kb0 + i);
        __syncwarp();
        issued = pre;
        uint32_t phase = 0;
        for (int i = pre, s = 0; i < n; ++i, ++issued) {
            if (!wait_all(smem_u32(&ctl->empty[s]), phase, abort_flag, g)) break;
            if (el) {
                weights(s, kb0 + i);
                tokens(s, kb0 + i);
            }
            __syncwarp();
            if (++s == S) { s = 0; phase ^= 1u; }
        }
    } else if (active && warp == 1) {
        const bool el = elected();
        const uint32_t idesc = idesc_f16_f32(128, BN);
        uint32_t phase = 0, aphase = 0;
        for (int i = 0, s = 0, a = 0; i < n; ++i) {
            const int chunk = i / kChunkBlocks, d = chunk % C::ND, in = i % kChunkBlocks;
            if (!wait_all(smem_u32(&ctl->full[s]), phase, abort_flag, g) ||
                !wait_all(smem_u32(&ctl->afull[a]), aphase, abort_flag, g) ||
                (in == 0 && !wait_all(smem_u32(&ctl->dempty[d]), (uint32_t)((chunk / C::ND) & 1) ^ 1u, abort_flag, g)))
                break;
            tc_fence_after();
            const uint32_t x = base + s * C::STAGE + kWeightTile;
            if (el) {
#pragma unroll
                for (int kk = 0; kk < kInner / 16; ++kk)
                    tc_mma_f16_ts(tmem_base + (uint32_t)(d * BN), tmem_a + (uint32_t)(a * kATmem + kk * 8),
                                  smem_desc_sw128(x + (kk / 4) * (C::TOKENS / 2)) + (uint64_t)(kk % 4 * 2), idesc,
                                  in > 0 || kk > 0 ? 1u : 0u);
                tc_commit(smem_u32(&ctl->empty[s]));
                tc_commit(smem_u32(&ctl->aempty[a]));
                if (in == kChunkBlocks - 1 || i == n - 1) tc_commit(smem_u32(&ctl->dfull[d]));
            }
            __syncwarp();
            if (++s == S) { s = 0; phase ^= 1u; }
            if (++a == C::NA) { a = 0; aphase ^= 1u; }
        }
    }

    int acc[C::CPT];
    const bool works = warp >= 2;
    const int q = warp & 3, row = q * 32 + lane, h = works ? (warp - 2) / 4 : 0, col0 = h * C::CPT;
    if (active && works) {
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const int chunks = (n + kChunkBlocks - 1) / kChunkBlocks;
#pragma unroll
        for (int c = 0; c < C::CPT; ++c) acc[c] = 0;
        bool ok = true;
        // A chunk's sums are read before the second k-block behind it is converted: the MMAs of that one would wait for them.
        for (int i = h, chunk = 0; ok; i += 2) {
            while (ok && chunk < chunks && ((chunk + 1) * kChunkBlocks + 2 <= i || i >= n)) {
                const int d = chunk % C::ND;
                ok = wait_all(smem_u32(&ctl->dfull[d]), (uint32_t)((chunk / C::ND) & 1), abort_flag, g);
                if (!ok) break;
                ++chunk;
                tc_fence_after();
                const uint32_t src = tmem_base + (uint32_t)(d * BN + col0) + lanes;
                constexpr int kLoad = C::CPT < 16 ? 8 : 16;
#pragma unroll
                for (int c = 0; c < C::CPT; c += kLoad) {
                    uint32_t v[kLoad];
                    if constexpr (kLoad == 8) tmem_ld8(src + c, v); else tmem_ld16(src + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < kLoad; ++j) acc[c + j] += __float2int_rn(__uint_as_float(v[j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->dempty[d]));
            }
            if (!ok || i >= n) break;
            const int s = i % S, a = i % C::NA;
            // In this order: the slot's wait says that the MMAs of k-block i - NA are done, and so that the stage's k-block before
            // this one, which the other warps may have converted, has landed: else its parity could be taken for this one's.
            ok = wait_all(smem_u32(&ctl->aempty[a]), (uint32_t)((i / C::NA) & 1) ^ 1u, abort_flag, g) &&
                 wait_all(smem_u32(&ctl->full[s]), (uint32_t)((i / S) & 1), abort_flag, g);
            if (!ok) break;
            tc_fence_after();
            convert_rows(ring + (size_t)s * C::STAGE, row, tmem_a + (uint32_t)(a * kATmem) + lanes);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->afull[a]));
        }
        __syncwarp();
    }

    // ---- the cluster's sums: every CTA gets a slice of the token columns from all, in groups of four: [part][group][row]
    int4 *red = reinterpret_cast<int4 *>(ring);
    const int slice = (BN / 4 + parts - 1) / parts;
    if (parts > 1) {
        cluster_sync();   // every ring of the cluster is idle
        if (active && works) {
#pragma unroll
            for (int c = 0; c < C::CPT; c += 4)
                if (col0 + c < t.rows) {
                    const int quad = (col0 + c) / 4, to = quad / slice, at = quad - to * slice;
                    st_cluster_s32x4(map_to_rank(smem_u32(red + (size_t)(part * slice + at) * 128 + row), (uint32_t)to),
                                     make_int4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]));
                }
        }
        cluster_sync();
    }
    if (active && works) {
        const int64_t out_n = (int64_t)m * 128 + row;
        if (out_n < g.N) {
            const float w = g.ws[(int64_t)t.group * g.N + out_n];
            auto store = [&](int col, int sum) {
                const float y = (float)sum * g.xs[t.row0 + col] * w;
                const int64_t at = (int64_t)(t.row0 + col) * g.N + out_n;
                if (g.out_f32)
                    static_cast<float *>(g.out)[at] = y;
                else
                    static_cast<uint16_t *>(g.out)[at] = f32_to_bf16_bits(y);
            };
            if (parts == 1) {
#pragma unroll
                for (int c = 0; c < C::CPT; ++c)
                    if (col0 + c < t.rows) store(col0 + c, acc[c]);
            } else {
                const int first = part * slice, mine = min(min(slice, BN / 4 - first), (t.rows + 3) / 4 - first);
                for (int at = h; at < mine; at += 2) {
                    int4 v = make_int4(0, 0, 0, 0);
                    for (int r = 0; r < parts; ++r) {
                        const int4 o = red[(size_t)(r * slice + at) * 128 + row];
                        v = make_int4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
                    }
                    const int col = (first + at) * 4, each[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (col + j < t.rows) store(col + j, each[j]);
                }
            }
        }
    }

    // ---- teardown: nothing in flight (after an abort: bounded waits), then the TMEM goes back
    if (warp == 0 && lane == 0) {
        for (int i = max(0, issued - S); i < issued; ++i)
            if (!mbar_wait_drain(smem_u32(&ctl->full[i % S]), (uint32_t)((i / S) & 1), drain_limit_of(g.wait_limit_ns)))
                __nanosleep(200000);
    }
    if (warp == 1 && lane == 0) {
        tc_commit(smem_u32(&ctl->drain));
        (void)mbar_wait_drain(smem_u32(&ctl->drain), 0, drain_limit_of(g.wait_limit_ns));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::TMEM);
}

template <typename C>
cudaError_t run(const CUtensorMap &tw, const CUtensorMap &tx, const Int8Gemm &g, int kb, int parts, int slots, int row_tiles,
                int stream_weights, bool whole, bool pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done;   // bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(done.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(int8_cols_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        done.fetch_or(1ull << (dev & 63), std::memory_order_acq_rel);
    }
    const int stages = whole ? C::WHOLE : C::PART;
    return launch_kernel(int8_cols_kernel<C>, dim3((unsigned)parts, (unsigned)slots, (unsigned)row_tiles), kColsThreads,
                         C::FIXED + (size_t)stages * C::STAGE, pdl, parts, s, tw, tx, g, kb, stream_weights, stages);
}

}  // namespace

// CTAs that share a tile's k-blocks: as many as find room, two on an SM (nearly), four k-blocks each at least.  (us with 1, 2, 3 and
// 4 parts: 16 x 12288 x 7168, 96 tiles, 24.6, 21.5, 21.1, 25.0; 64 x 12288 x 7168 28.7, 27.5, 26.1, 29.3; 16 x 2112 x 7168, 17 tiles,
// 21.6, 14.2, .., 10.5, and with eight 9.9; 64 x 7168 x 6144, 56 tiles, 23.5, 19.6, .., 16.4.)
int int8_cols_parts(int64_t tiles, int kb, int sm_count) {
    const int64_t room = std::min<int64_t>(19 * (int64_t)sm_count / 10 / std::max<int64_t>(1, tiles), kb / 4);
    return (int)std::min<int64_t>(std::max<int64_t>(room, 1), 16 * tiles <= sm_count && kb >= 24 ? 8 : 5);
}

// grouped: every group may begin a tile of its own; as many as there are rows at most
int64_t int8_cols_slots(const Int8Gemm &g, int tile_rows) {
    return g.offsets ? std::min<int64_t>(g.T, g.T / tile_rows + std::min<int64_t>(g.groups, g.T)) : (g.T + tile_rows - 1) / tile_rows;
}

mse_status launch_int8_cols(const Int8Gemm &g, int tile_rows, int sm_count, bool pdl, cudaStream_t s) {
    CUtensorMap tw, tx;
    mse_status st = map_bytes(&tw, g.wq, g.groups * g.N, g.K, g.ldw, 128);
    if (st != MSE_OK) return st;
    if ((st = map_bytes(&tx, g.x16, g.T, g.K * 2, g.ldx16 * 2, tile_rows)) != MSE_OK) return st;
    const int kb = (int)((g.K + kInner - 1) / kInner);
    const int64_t row_tiles = (g.N + 127) / 128, slots = int8_cols_slots(g, tile_rows);
    if (row_tiles > 65535 || slots > 65535) return MSE_ERR_UNSUPPORTED_SHAPE;
    const int parts = int8_cols_parts(row_tiles * slots, kb, sm_count);
    const int stream_weights = slots == 1 || (g.offsets && g.T <= (int64_t)tile_rows * g.groups);
    const bool whole = parts == 1 && row_tiles * slots <= sm_count;
    cudaError_t e;
    auto with = [&](auto c) {
        return run<decltype(c)>(tw, tx, g, kb, parts, (int)slots, (int)row_tiles, stream_weights, whole, pdl, s);
    };
    switch (tile_rows) {
        case 16: e = with(Cols<16>()); break;
        case 32: e = with(Cols<32>()); break;
        default: e = with(Cols<64>()); break;
    }
    return e == cudaSuccess ? MSE_OK : MSE_ERR_CUDA;
}

}  // namespace sorted
}  // namespace mse
