// Block-scaled 8-bit product for few token rows: weights fill the 128-row side of the MMA,
// up to 64 tokens are its columns (swap-AB), so that a weight byte is read once and no MMA
// row is padding.
//
// out[n, t] = sum_b ws[n / 128, b] xs[t, b] (sum_{k in b} w[n, k] x[t, k]).  A scale of one
// k-block multiplies a sum over 128 products, so the tensor cores sum one k-block at a time
// into a fresh TMEM buffer (2 or 4 of them in turn), and the promotion warps add it, scaled,
// to fp32 sums in registers.  A CTA owns one 128-row weight tile (SWIGLU: gate and up tile)
// and one token tile; the k-blocks may be split over a cluster, whose CTAs exchange their
// sums through distributed shared memory and each finish a slice of the token columns, in
// rank order.
//
// Warp 0 loads (TMA), warp 1 issues MMAs, the others promote (and, for a few tokens in bf16, round them).
#include <atomic>

#include "device.h"
#include "fp8_tc.cuh"
#include "launch.h"

namespace mse {
namespace routed {
namespace {

constexpr int kChunk = 32;       // k-blocks whose scales are in shared memory at a time
constexpr int kMaxColsStages = 9;
constexpr int kXsRing = 16;      // k-blocks of token scales, where the kernel rounds the tokens itself
constexpr int kRoundQuads = kRoundRows / 4;

constexpr int pow2_up(int v) {
    int p = 32;
    while (p < v) p <<= 1;
    return p;
}

struct ColsCtrl {
    uint64_t full[kMaxColsStages], empty[kMaxColsStages], tfull[4], tempty[4], xs_full[kXsRing], drain;
    uint32_t tmem_base;
    int abort_flag;
};

// ROUND: the tokens come in bf16, and four more warps round them to 8 bits, each every fourth k-block, straight into
// the ring: up to kRoundRows tokens of a plain product need no launch of their own for that.
template <int BN_, int EPI_, bool ROUND_ = false>
struct Cols {
    static constexpr int BN = BN_, EPI = EPI_;
    static constexpr bool ROUND = ROUND_;
    static constexpr int ROUND_WARPS = ROUND ? 4 : 0;
    static_assert(!ROUND || (BN == 16 && EPI != BLOCK_SWIGLU), "a plain product of few tokens");
    // slot i mod kXsRing is written again only when the promotion is past it: the ring and the TMEM buffers bound
    // how far it lags
    static_assert(!ROUND || kMaxColsStages + 4 < kXsRing, "scales");
    static constexpr int MATS = EPI == BLOCK_SWIGLU ? 2 : 1;
    // Promotion: two groups of four warps.  Up to 32 columns of one product they take k-blocks in turn and halve
    // the columns at the end; with 64, or gate and up, each takes half of them throughout (us by k-blocks and by
    // columns: 32 x 4096 x 2048 7.8 and 8.6, 16 x 12288 x 7168 18.9 and 19.6, 64 x 12288 x 7168 23.7 and 22.4; experts of 128 tokens
    // 289 and 283).  Gate and up of 16 columns are one group's (two by k-blocks: a decode batch's experts 210 us, 202).
    static constexpr bool BY_K = BN < 64 && MATS == 1;
    static constexpr int GROUPS = BN * MATS == 32 && !BY_K ? 1 : 2, WARPS = 4 * GROUPS;
    static constexpr int CPT = BN / GROUPS;                    // token columns a thread finishes
    static constexpr int ACC = BY_K ? BN : CPT;                // and sums
    static_assert(ACC % 16 == 0, "TMEM loads of 16 columns");
    static constexpr int THREADS = 64 + 32 * (WARPS + ROUND_WARPS);
    static constexpr int BUF = MATS * BN;                      // TMEM columns of one k-block's sums
    static constexpr int NBUF = BUF * 4 <= 256 ? 4 : 2;
    static constexpr int TMEM = pow2_up(NBUF * BUF);
    static constexpr int CTAS = 2;                             // resident per SM (the ring may take a whole SM)
    static_assert(CTAS * TMEM <= 512, "TMEM");
    static constexpr uint32_t STAGE = MATS * kOperandTile + BN * 128;
    static constexpr int XS_PITCH = BN + 4;                    // floats; 16-byte rows, 4-way conflicts at worst
    static constexpr uint32_t SCALES = kChunk * XS_PITCH * 4 + MATS * kChunk * 4 + 4 * BN * 4;
    static constexpr uint32_t FIXED = 1024 + SCALES + sizeof(ColsCtrl) + 64;
    // stages of the ring with two CTAs on an SM, or one
    static constexpr int fit(uint32_t budget) {
        const int n = (int)((budget - FIXED) / STAGE);
        return n < kMaxColsStages ? n : kMaxColsStages;
    }
    static constexpr int HALF = fit(113 * 1024), WHOLE = fit(227 * 1024);
    static_assert(HALF >= 2, "ring");
    // the groups' halves, and the exchange of a split tile (at most BN / 4 + 7 groups of four columns), use the ring
    static_assert(MATS * BN * 512 <= HALF * STAGE, "halves");
    static_assert(MATS * (BN / 4 + 7) * 2048 <= HALF * STAGE, "exchange");
};

// The token tile of slot z of a dispatch of at most 32 pairs, from the ids themselves: experts ascending, tiles
// of tile_rows rows.  Every warp finds it alone.
__device__ __forceinline__ bool tile_of_ids(const BlockGemm &g, int z, int lane, Tile &t) {
    const int64_t e64 = lane < g.pairs ? (int64_t)g.ids[lane] - g.first_expert : -1;
    const int e = e64 >= 0 && e64 < g.groups ? (int)e64 : -1;
    const uint32_t same = __match_any_sync(~0u, e);
    const int count = e < 0 ? 0 : __popc(same), tiles = (count + g.tile_rows - 1) / g.tile_rows;
    const bool head = e >= 0 && lane == __ffs(same) - 1;
    int rows_before = 0, tiles_before = 0;
    for (int j = 0; j < 32; ++j) {   // the experts before this one, each counted at its first pair
        const int eo = __shfl_sync(~0u, head ? e : -1, j), co = __shfl_sync(~0u, count, j),
                  to = __shfl_sync(~0u, tiles, j);
        if (eo >= 0 && eo < e) { rows_before += co; tiles_before += to; }
    }
    const uint32_t owner = __ballot_sync(~0u, head && z >= tiles_before && z < tiles_before + tiles);
    if (owner == 0) return false;
    const int from = __ffs(owner) - 1, skip = (z - __shfl_sync(~0u, tiles_before, from)) * g.tile_rows;
    t.row0 = __shfl_sync(~0u, rows_before, from) + skip;
    t.rows = min(g.tile_rows, __shfl_sync(~0u, count, from) - skip);
    t.expert = __shfl_sync(~0u, e, from);
    return true;
}

template <typename C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    cols_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const BlockGemm g,
                const int stream_weights, const int S) {
    constexpr int BN = C::BN, MATS = C::MATS, CPT = C::CPT;
    constexpr int kPromo = 32 * C::WARPS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *ring = smem_raw + (base - raw);
    float *xs_s = reinterpret_cast<float *>(ring + (size_t)S * C::STAGE);   // [kChunk][XS_PITCH]
    float *ws_s = xs_s + kChunk * C::XS_PITCH;                              // [MATS][kChunk]
    uint32_t *amax_s = reinterpret_cast<uint32_t *>(ws_s + MATS * kChunk);  // [4][BN]
    ColsCtrl *ctl = reinterpret_cast<ColsCtrl *>(amax_s + 4 * BN);
    const int warp = __shfl_sync(~0u, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int part = blockIdx.x, parts = gridDim.x, m = blockIdx.z;
    const int kb0 = (int)((int64_t)g.kb * part / parts), n = (int)((int64_t)g.kb * (part + 1) / parts) - kb0;
    volatile int *abort_flag = &ctl->abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), C::ROUND ? 2 : 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        if constexpr (C::ROUND)
            for (int i = 0; i < kXsRing; ++i) mbar_init(smem_u32(&ctl->xs_full[i]), 1);
        for (int b = 0; b < C::NBUF; ++b) {
            mbar_init(smem_u32(&ctl->tfull[b]), 1);
            mbar_init(smem_u32(&ctl->tempty[b]), C::BY_K ? C::WARPS / 2 : C::WARPS);
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
    const uint32_t tmem_base = __shfl_sync(~0u, ctl->tmem_base, 0);
    // weights_early: the tile table (or the ids) and the weights were complete before this launch could start, and
    // only the tokens and their scales are the previous kernel's
    if (!g.weights_early) pdl_wait();
    Tile t;
    const bool active = g.ids ? tile_of_ids(g, blockIdx.y, lane, t) : tile_of_slot(g, blockIdx.y, t);
    // Only now may the next kernel of the layer start: what it reads before its own wait is complete.  (With ids the
    // table is not, until the wait is over.  A call's last kernel lets nothing start early: its outputs may be
    // anything to the next one.)
    if (g.tiles && !g.ids) pdl_launch_dependents();
    // A grid without a tile (slot 0 has none) waits too: it would else be over before the kernel before it, and the next call
    // would write the tile table under that one's eyes.  With tiles, the CTAs that have one wait for all.
    if (!active && (g.ids || (g.weights_early && blockIdx.y == 0))) pdl_wait();

    const int w_row = active ? (int)(t.expert * g.w_group_rows) + m * kBlock : 0;
    int issued = 0;
    if (active && warp == 0) {
        const bool el = elect_lane();
        const uint64_t pol_w = stream_weights ? l2_policy_evict_first() : l2_policy_evict_last();
        const uint64_t pol_x = l2_policy_evict_last();
        auto weights = [&](int s, int kb) {
            const uint32_t bar = smem_u32(&ctl->full[s]), dst = base + s * C::STAGE;
            mbar_arrive_expect_tx(bar, C::ROUND ? MATS * kOperandTile : C::STAGE);
            tma_load_2d(dst, &tmW, bar, kb * kBlock, w_row, pol_w);
            if constexpr (MATS == 2)
                tma_load_2d(dst + kOperandTile, &tmW, bar, kb * kBlock, w_row + (int)g.up_rows, pol_w);
        };
        auto tokens = [&](int s, int kb) {
            if constexpr (!C::ROUND) tma_load_2d(base + s * C::STAGE + MATS * kOperandTile, &tmX, smem_u32(&ctl->full[s]), kb * kBlock, t.row0,
                        pol_x);
        };
        const int pre = min(S, n);
        for (int i = 0; i < pre; ++i)
            if (el) weights(i, kb0 + i);
        if (g.weights_early) pdl_wait();
        if (g.ids) pdl_launch_dependents();
        for (int i = 0; i < pre; ++i)
            if (el) tokens(i, kb0 + i);
        __syncwarp();
        issued = pre;
        uint32_t phase = 0;
        for (int i = pre, s = 0; i < n; ++i, ++issued) {
            if (!warp_wait(smem_u32(&ctl->empty[s]), phase, abort_flag, g)) break;
            if (el) {
                weights(s, kb0 + i);
                tokens(s, kb0 + i);
            }
            __syncwarp();
            if (++s == S) { s = 0; phase ^= 1u; }
        }
    } else if (active && warp == 1) {
        const bool el = elect_lane();
        const uint32_t idesc = idesc_e4m3_f32(128, BN);
        uint32_t phase = 0;
        for (int i = 0, s = 0; i < n; ++i) {
            const int b = i % C::NBUF;
            if (!warp_wait(smem_u32(&ctl->full[s]), phase, abort_flag, g) ||
                !warp_wait(smem_u32(&ctl->tempty[b]), (uint32_t)((i / C::NBUF) & 1) ^ 1u, abort_flag, g))
                break;
            tc_fence_after();
            const uint32_t st = base + s * C::STAGE;
            const uint64_t xd = smem_desc_sw128(st + MATS * kOperandTile);
            if (el) {
#pragma unroll
                for (int a = 0; a < MATS; ++a) {
                    const uint64_t wd = smem_desc_sw128(st + a * kOperandTile);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_e4m3(tmem_base + (uint32_t)(b * C::BUF + a * BN), wd + (uint64_t)(kk * 2),
                                    xd + (uint64_t)(kk * 2), idesc, kk > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(&ctl->tfull[b]));
                tc_commit(smem_u32(&ctl->empty[s]));
            }
            __syncwarp();
            if (++s == S) { s = 0; phase ^= 1u; }
        }
    }

    if constexpr (C::ROUND) {
        if (active && warp >= 2 + C::WARPS) {
            // Warp w of the four: k-blocks w, w + 4, ..; 8 lanes for a token, 16 values each, four tokens at a time.
            // The values of its next k-block are on their way while this one's are rounded.
            const int first = warp - 2 - C::WARPS, sub = lane % 8;
            auto fetch = [&](int i, int quad, uint32_t (&to)[8]) {
                const int token = quad * 4 + lane / 8;
                const int64_t k = (int64_t)(kb0 + i) * kBlock + sub * 16;
                const uint16_t *x = g.x + (int64_t)(t.row0 + token) * g.ldxb + k;
#pragma unroll
                for (int v = 0; v < 8; ++v) to[v] = 0;
                if (i >= n || token >= t.rows) return;
                if (g.x_wide && k + 16 <= g.K) {
                    const uint4 lo = *reinterpret_cast<const uint4 *>(x);
                    const uint4 hi = reinterpret_cast<const uint4 *>(x)[1];
                    to[0] = lo.x; to[1] = lo.y; to[2] = lo.z; to[3] = lo.w;
                    to[4] = hi.x; to[5] = hi.y; to[6] = hi.z; to[7] = hi.w;
                } else {
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const uint32_t a = k + 2 * v < g.K ? x[2 * v] : 0u;
                        const uint32_t b = k + 2 * v + 1 < g.K ? x[2 * v + 1] : 0u;
                        to[v] = a | (b << 16);
                    }
                }
            };
            uint32_t next[kRoundQuads][8];
#pragma unroll
            for (int quad = 0; quad < kRoundQuads; ++quad)
                if (quad * 4 < t.rows) fetch(first, quad, next[quad]);
            bool ok = true;
            for (int i = first; i < n && ok; i += C::ROUND_WARPS) {
                const int s = i % S, slot = i % kXsRing;
                ok = warp_wait(smem_u32(&ctl->empty[s]), (uint32_t)((i / S) & 1) ^ 1u, abort_flag, g);
                if (!ok) break;
#pragma unroll
                for (int quad = 0; quad < kRoundQuads; ++quad) {
                    if (quad * 4 >= t.rows) break;
                    uint32_t now[8], top = 0, w[4];
#pragma unroll
                    for (int v = 0; v < 8; ++v) now[v] = next[quad][v];
                    fetch(i + C::ROUND_WARPS, quad, next[quad]);
#pragma unroll
                    for (int v = 0; v < 8; ++v) top = abs_max2(top, now[v]);
#pragma unroll
                    for (int d = 4; d > 0; d >>= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, d));
                    const float a = floored_amax(bits_of_max2(top));
                    const E4m3Scale scale = e4m3_scale(a);
#pragma unroll
                    for (int v = 0; v < 4; ++v) w[v] = e4m3x4(now[2 * v], now[2 * v + 1], scale);
                    const int token = quad * 4 + lane / 8;
                    // the 128-byte swizzle of the operand tiles: 16-byte word `sub` of a row at sub ^ (row mod 8)
                    *reinterpret_cast<uint4 *>(ring + (size_t)s * C::STAGE + MATS * kOperandTile + token * 128 +
                                               ((sub ^ (token & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (sub == 0) xs_s[slot * C::XS_PITCH + token] = block_scale(a);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&ctl->full[s]));
                    mbar_arrive(smem_u32(&ctl->xs_full[slot]));
                }
            }
            __syncwarp();
        }
    }

    float acc[MATS][CPT];
    const bool promo = warp >= 2 && warp < 2 + C::WARPS;
    const int q = warp & 3, row = q * 32 + lane, group = promo ? (warp - 2) / 4 : 0, col0 = group * CPT;
    if (active && promo) {
        float sum[MATS][C::ACC];
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
            for (int c = 0; c < C::ACC; ++c) sum[a][c] = 0.f;
        if (g.weights_early) pdl_wait();
        const int pt = threadIdx.x - 64;
        const float *ws = g.ws + (int64_t)t.expert * g.ws_group + (int64_t)m * g.kb;
        bool ok = true;
        for (int c0 = 0; c0 < n; c0 += kChunk) {
            // (a warp whose wait ran out takes the others along: nobody is left at a barrier)
            if (c0 > 0 && !named_barrier_and(1, kPromo, ok)) break;
            if constexpr (!C::ROUND) {
                // (all loads before the first store: one trip to L2, not one for each)
                constexpr int kPer = kChunk * BN / kPromo;
                float v[kPer];
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int i = pt + u * kPromo, k = i % kChunk, j = i / kChunk;
                    v[u] = j < t.rows && c0 + k < n ? __ldcg(g.xs + (int64_t)(t.row0 + j) * g.kb + kb0 + c0 + k) : 0.f;
                }
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int i = pt + u * kPromo;
                    xs_s[i % kChunk * C::XS_PITCH + i / kChunk] = v[u];
                }
            }
            if (pt < MATS * kChunk && c0 + pt % kChunk < n)
                ws_s[pt] = ws[(pt / kChunk) * g.up_scales + kb0 + c0 + pt % kChunk];
            named_barrier_sync(1, kPromo);
            for (int k = C::BY_K ? group : 0; k < kChunk && c0 + k < n; k += C::BY_K ? 2 : 1) {   // kChunk is even
                const int i = c0 + k, b = i % C::NBUF;
                ok = warp_wait(smem_u32(&ctl->tfull[b]), (uint32_t)((i / C::NBUF) & 1), abort_flag, g);
                if constexpr (C::ROUND)
                    ok = ok && warp_wait(smem_u32(&ctl->xs_full[i % kXsRing]), (uint32_t)((i / kXsRing) & 1), abort_flag, g);
                if (!ok) break;
                tc_fence_after();
                const float *x = xs_s + (C::ROUND ? i % kXsRing : k) * C::XS_PITCH + (C::BY_K ? 0 : col0);
                const uint32_t src = tmem_base + (uint32_t)(b * C::BUF + (C::BY_K ? 0 : col0)) + ((uint32_t)(q * 32) << 16);
#pragma unroll
                for (int c = 0; c < C::ACC; c += 16) {
                    uint32_t d[MATS][16];
#pragma unroll
                    for (int a = 0; a < MATS; ++a) tmem_ld16(src + a * BN + c, d[a]);
                    tmem_ld_wait();
#pragma unroll
                    for (int a = 0; a < MATS; ++a) {
                        const float w = ws_s[a * kChunk + k];
#pragma unroll
                        for (int v = 0; v < 16; v += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(x + c + v);
                            sum[a][c + v] = fmaf(__uint_as_float(d[a][v]), f.x * w, sum[a][c + v]);
                            sum[a][c + v + 1] = fmaf(__uint_as_float(d[a][v + 1]), f.y * w, sum[a][c + v + 1]);
                            sum[a][c + v + 2] = fmaf(__uint_as_float(d[a][v + 2]), f.z * w, sum[a][c + v + 2]);
                            sum[a][c + v + 3] = fmaf(__uint_as_float(d[a][v + 3]), f.w * w, sum[a][c + v + 3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[b]));
            }
        }
        __syncwarp();
        if constexpr (C::BY_K) {
            // every MMA is done: the ring takes the halves that the groups owe one another, [group][mat][column][row]
            named_barrier_sync(1, kPromo);
            float *owed = reinterpret_cast<float *>(ring);
#pragma unroll
            for (int a = 0; a < MATS; ++a)
#pragma unroll
                for (int c = 0; c < CPT; ++c)
                    if (c + CPT - col0 < t.rows)
                        owed[((group * MATS + a) * CPT + c) * 128 + row] = group == 0 ? sum[a][CPT + c] : sum[a][c];
            named_barrier_sync(1, kPromo);
#pragma unroll
            for (int a = 0; a < MATS; ++a)
#pragma unroll
                for (int c = 0; c < CPT; ++c)   // group 0's sum first in either half
                    acc[a][c] = col0 + c >= t.rows ? 0.f
                                : group == 0       ? sum[a][c] + owed[((MATS + a) * CPT + c) * 128 + row]
                                                   : owed[(a * CPT + c) * 128 + row] + sum[a][CPT + c];
        } else {
#pragma unroll
            for (int a = 0; a < MATS; ++a)
#pragma unroll
                for (int c = 0; c < CPT; ++c) acc[a][c] = sum[a][c];
        }
    }

    // ---- the cluster's sums: every CTA gets a slice of the token columns from all, in groups of four columns:
    // [rank][mat][group][row] (16-byte stores: 4-byte ones made the exchange of 64 columns 4 us long)
    float4 *red = reinterpret_cast<float4 *>(ring);
    const int slice = (BN / 4 + parts - 1) / parts;
    if (parts > 1) {
        cluster_sync();   // every ring of the cluster is idle
        if (active && promo) {
#pragma unroll
            for (int c = 0; c < CPT; c += 4) {
                const int quad = (col0 + c) / 4;
                if (quad * 4 < t.rows) {
                    const int to = quad / slice, at = quad - to * slice;
#pragma unroll
                    for (int a = 0; a < MATS; ++a)
                        st_cluster_f32x4(map_to_rank(smem_u32(red + (size_t)((part * MATS + a) * slice + at) * 128 + row),
                                                     (uint32_t)to),
                                         make_float4(acc[a][c], acc[a][c + 1], acc[a][c + 2], acc[a][c + 3]));
                }
            }
        }
        cluster_sync();
    }
    if (active && promo) {
        const int64_t out_n = (int64_t)m * kBlock + row;
        const bool valid = out_n < g.N;
        auto summed = [&](int a, int at) {   // in rank order
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < parts; ++r) {
                const float4 o = red[(size_t)((r * MATS + a) * slice + at) * 128 + row];
                v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            return v;
        };
        const int first = part * slice;                                              // parts > 1: this CTA's groups of
        const int mine = min(min(slice, BN / 4 - first), (t.rows + 3) / 4 - first);  // columns
        // (this group's: every GROUPS-th from `group` on)
        if constexpr (C::EPI != BLOCK_SWIGLU) {
            auto store = [&](int col, float v) {
                const int64_t at = (int64_t)(t.row0 + col) * g.ldo + out_n;
                if constexpr (C::EPI == BLOCK_BF16)
                    static_cast<uint16_t *>(g.out)[at] = f32_to_bf16_bits(v);
                else
                    static_cast<float *>(g.out)[at] = v;
            };
            if (valid) {
                if (parts == 1) {
#pragma unroll
                    for (int c = 0; c < CPT; ++c)
                        if (col0 + c < t.rows) store(col0 + c, acc[0][c]);
                } else {
                    for (int at = group; at < mine; at += C::GROUPS) {
                        const float4 v = summed(0, at);
                        const float each[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if ((first + at) * 4 + j < t.rows) store((first + at) * 4 + j, each[j]);
                    }
                }
            }
        } else {
            // h = silu(g) u; the largest |h| of a token over the tile's 128 rows is its block's scale
            auto h_of = [&](float gate, float up) { return valid ? glu(gate, up) : 0.f; };
            auto note = [&](int col, float h) {
                const uint32_t a = __reduce_max_sync(~0u, abs_bits(h));
                if (lane == 0) amax_s[q * BN + col] = a;
            };
            auto write = [&](int col, float h) {
                const float a = floored_amax(max(max(amax_s[col], amax_s[BN + col]),
                                                 max(amax_s[2 * BN + col], amax_s[3 * BN + col])));
                const int64_t r = t.row0 + col;
                if (valid) g.hq[r * g.ldh + out_n] = e4m3_of(h, a, __frcp_rn(a));
                if (row == 0) g.hs[r * g.hb + m] = block_scale(a);
            };
            if (parts == 1) {
#pragma unroll
                for (int c = 0; c < CPT; ++c)
                    if (col0 + c < t.rows) {
                        acc[0][c] = h_of(acc[0][c], acc[MATS - 1][c]);
                        note(col0 + c, acc[0][c]);
                    }
                named_barrier_sync(1, kPromo);
#pragma unroll
                for (int c = 0; c < CPT; ++c)
                    if (col0 + c < t.rows) write(col0 + c, acc[0][c]);
            } else {
                for (int at = group; at < mine; at += C::GROUPS) {
                    const float4 gate = summed(0, at), up = summed(MATS - 1, at);
                    const float4 h = make_float4(h_of(gate.x, up.x), h_of(gate.y, up.y), h_of(gate.z, up.z),
                                                 h_of(gate.w, up.w));
                    red[(size_t)at * 128 + row] = h;             // read again by this thread alone
                    const float each[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) note((first + at) * 4 + j, each[j]);
                }
                named_barrier_sync(1, kPromo);
                for (int at = group; at < mine; at += C::GROUPS) {
                    const float4 h = red[(size_t)at * 128 + row];
                    const float each[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((first + at) * 4 + j < t.rows) write((first + at) * 4 + j, each[j]);
                }
            }
        }
    }

    // ---- teardown: nothing in flight (after an abort: bounded waits), then the TMEM goes back
    if (warp == 0 && lane == 0) {
        for (int i = max(0, issued - S); i < issued; ++i)
            if (!mbar_wait_drain(smem_u32(&ctl->full[i % S]), (uint32_t)((i / S) & 1), drain_limit(g.wait_limit_ns)))
                __nanosleep(200000);
    }
    if (warp == 1 && lane == 0) {
        tc_commit(smem_u32(&ctl->drain));
        (void)mbar_wait_drain(smem_u32(&ctl->drain), 0, drain_limit(g.wait_limit_ns));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::TMEM);
}

template <typename C>
cudaError_t run(const CUtensorMap &tw, const CUtensorMap &tx, const BlockGemm &g, int parts, int slots, int row_tiles,
                int stream_weights, bool whole, bool pdl, cudaStream_t s) {
    static std::atomic<uint64_t> done;   // bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(done.load(std::memory_order_acquire) >> (dev & 63) & 1)) {
        e = cudaFuncSetAttribute(cols_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        done.fetch_or(1ull << (dev & 63), std::memory_order_acq_rel);
    }
    const int stages = whole ? C::WHOLE : C::HALF;
    return launch_kernel(cols_kernel<C>, dim3((unsigned)parts, (unsigned)slots, (unsigned)row_tiles), C::THREADS,
                         C::FIXED + (size_t)stages * C::STAGE, pdl, parts, s, tw, tx, g, stream_weights, stages);
}

template <int EPI>
cudaError_t run_bn(const CUtensorMap &tw, const CUtensorMap &tx, const BlockGemm &g, int parts, int slots,
                   int row_tiles, int stream_weights, bool whole, bool pdl, cudaStream_t s) {
    auto with = [&](auto c) {
        return run<decltype(c)>(tw, tx, g, parts, slots, row_tiles, stream_weights, whole, pdl, s);
    };
    if constexpr (EPI != BLOCK_SWIGLU) {
        if (g.tile_rows == 64) return with(Cols<64, EPI>());
        if (g.x) return with(Cols<16, EPI, true>());
    }
    return g.tile_rows == 16 ? with(Cols<16, EPI>()) : with(Cols<32, EPI>());
}

}  // namespace

// CTAs that share a tile's k-blocks.
// One SM's loads bring a k-block every 0.2 to 0.3 us, so a tile's k-blocks are split over as many CTAs as find
// room, two on an SM (nearly: clusters do not fill every last place, and one that waits doubles the time), down to
// two k-blocks each: up to five parts (larger clusters find fewer places), eight
// where there are few tiles.  (us with 1, 3, 4, 5, 6 and 8 parts: 64 x 12288 x 7168, 96 tiles, 23.5, 19.2, 24.6, ..;
// 64 x 7168 x 6144, 56 tiles, 20.1, 14.3, 13.4, 13.6, 18.1, 19.8; 64 x 2048 x 2048, 16 tiles, 9.3, 7.0, 6.4, 6.5, 6.1, 7.5;
// 200 x 700 x 1200, 24 tiles, 8.3, 6.8, 6.4, 6.0, 6.8, 7.8; 16 x 1024 x 4096, 8 tiles, 10.7, 7.7, 7.1, 6.9, 6.7, 5.9;
// 64 x 7168 x 768, 56 tiles of six k-blocks, 5.9, 7.9.)
// Gate and up have twice the k-block: four of them at least, and of 32 tokens three CTAs on two SMs.  (The experts' layer with 1, 2,
// 3, 4 and 5 parts: 8 experts of 1024 x 896, 43 rows, 91 tiles of 8 k-blocks, 23.4, 22.0, 26.8, 26.9, 30.3; 4 of 4096 x 1024,
// 25 rows, 56 tiles of 32 k-blocks, 34.4, 29.8, 27.4, 26.6, 30.9; 8 of 2048 x 1536, 32 rows, 144 tiles, 30.3, 34.7, ..; the
// same with 16 rows 27.1, 26.1, 29.9; 8 of 1024 x 896, 15 rows, 77 tiles, 19.9, 18.7, 20.3.)
int cols_parts(int64_t tiles, int kb, int tile_rows, int epi, int sm_count) {
    const bool glu = epi == BLOCK_SWIGLU;
    const int64_t ctas = (glu && tile_rows > 16 ? 15 : 19) * (int64_t)sm_count / 10;
    const int64_t room = std::min<int64_t>(ctas / std::max<int64_t>(1, tiles), kb < 8 ? 1 : kb / (glu ? 4 : 2));
    const int parts = (int)std::min<int64_t>(std::max<int64_t>(room, 1), 16 * tiles <= sm_count && kb >= 24 ? 8 : 5);
    // 16 tokens take less time than the cluster where the tiles already fill most SMs (16 x 12288 x 7168 17.7 us whole,
    // 18.5 in three parts); gate and up of 16 have two operand tiles for it.
    return parts < 4 && tile_rows == 16 && !glu ? 1 : parts;
}

namespace {
int64_t cols_slots(const BlockGemm &g) { return g.tiles ? g.max_tiles : (g.T + g.tile_rows - 1) / g.tile_rows; }
int64_t cols_expected(const BlockGemm &g) {   // tiles of the whole grid, as far as the host can tell
    return blocks_of(g.N) * (g.tiles ? std::min<int64_t>(cols_slots(g), g.expected_tiles) : cols_slots(g));
}
}  // namespace

Split cols_split(const BlockGemm &g, int sm_count) {
    const int parts = cols_parts(cols_expected(g), g.kb, g.tile_rows, g.epi, sm_count);
    return {parts * cols_slots(g) * blocks_of(g.N), parts};
}

mse_status launch_block_cols(const BlockGemm &g, int sm_count, bool pdl, cudaStream_t s) {
    CUtensorMap tw, tx;
    mse_status st = map_bytes(&tw, g.wq, g.groups * g.w_group_rows, g.K, g.ldw, kBlock);
    if (st != MSE_OK) return st;
    if (g.x)
        tx = tw;   // the kernel rounds x itself
    else if ((st = map_bytes(&tx, g.xq, g.T, g.K, g.ldx, g.tile_rows)) != MSE_OK)
        return st;
    const int64_t row_tiles = blocks_of(g.N), slots = cols_slots(g);
    if (row_tiles > 65535 || slots > 65535) return MSE_ERR_UNSUPPORTED_SHAPE;
    const int parts = cols_split(g, sm_count).parts;
    const int stream_weights = g.tiles ? g.T <= (int64_t)g.tile_rows * g.groups : slots == 1;
    // one CTA per SM: its ring gets all of it (not in clusters, of which fewer would fit)
    const bool whole = parts == 1 && cols_expected(g) <= sm_count;
    cudaError_t e;
    switch (g.epi) {
        case BLOCK_BF16: e = run_bn<BLOCK_BF16>(tw, tx, g, parts, (int)slots, (int)row_tiles, stream_weights, whole, pdl, s); break;
        case BLOCK_F32: e = run_bn<BLOCK_F32>(tw, tx, g, parts, (int)slots, (int)row_tiles, stream_weights, whole, pdl, s); break;
        default: e = run_bn<BLOCK_SWIGLU>(tw, tx, g, parts, (int)slots, (int)row_tiles, stream_weights, whole, pdl, s); break;
    }
    return e == cudaSuccess ? MSE_OK : MSE_ERR_CUDA;
}

}  // namespace routed
}  // namespace mse
